"""Chunk attention over a paged cache against its definition in 64 bits."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case, attend

pytestmark = pytest.mark.gpu


def check(c, **kw):
    out, lse = c.attend(sda, **kw)
    torch.cuda.synchronize()
    ro, rl, to, tl = attend(c)
    rows = slice(c.q_indptr_l[0], c.q_indptr_l[-1])
    o, z, ro, rl = out.double().cpu()[rows], lse.double().cpu()[rows], ro[rows], rl[rows]
    assert torch.equal(torch.isnan(o), torch.isnan(ro))
    assert torch.equal(torch.isnan(z), torch.isnan(rl))
    fine = ~torch.isnan(ro)
    assert bool(((o - ro).abs() <= to[rows])[fine].all()), float(((o - ro).abs() - to[rows])[fine].max())
    both = torch.isinf(rl)
    assert torch.equal(z[both], rl[both])
    fine = torch.isfinite(rl)
    assert bool(((z - rl).abs() <= tl[rows])[fine].all()), float(((z - rl).abs() - tl[rows])[fine].max())
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 64, 128])
def test_shapes(D, H):
    check(Case(D + H, m=[1, 3, 0, 7], n=[70, 3, 200, 131], H=H, D=D, K=16))


@pytest.mark.parametrize("K", [1, 3, 16, 64, 100, 128])
def test_block_sizes(K):
    check(Case(K, m=[1, 1, 5, 40], n=[1, 64, 65, 300], H=16, D=512, K=K, base=5))


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 1000, 5000])
def test_one_token(n):
    check(Case(n, m=[1], n=[n], H=16, D=512, K=64))
    check(Case(n, m=[1] * 3, n=[n, 1, max(1, n // 2)], H=64, D=512, K=1))


@pytest.mark.parametrize("m,n", [([33], [33]), ([64], [640]), ([129], [1000]), ([200, 1, 17], [200, 900, 18])])
def test_chunks(m, n):
    check(Case(sum(n), m=m, n=n, H=8, D=512, K=64))


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (7, 4), (64, 0), (64, 64), (65, 70), (100, 3),
                                          (128, 200), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_window(window, first):
    check(Case(window % 977, m=[1, 90, 13], n=[500, 301, 13], H=16, D=128, K=16, window=window, first=first))
    check(Case(first % 977, m=[40], n=[700], H=16, D=512, K=64, window=window, first=first))


# Which kernel: at most 16 rows a sequence on average, at most 128, more (two CTAs work
# on 128 rows); K = 16: boxes of rows by TMA, K = 3: rows one by one.
KERNELS = [(4, 1, 16), (4, 1, 3), (64, 1, 16), (64, 1, 3), (64, 5, 16), (64, 5, 3)]


@pytest.mark.parametrize("H,m,K", KERNELS)
@pytest.mark.parametrize("D", [256, 512])
def test_rising_scores(H, m, K, D):
    """Rows whose scores exceed all before them by far: the running reference rises,
    O is scaled, in one row tile or the other, in several tiles of a piece."""
    n = 700
    loud = [(0, 70, 4.0), (0, 200, 9.0), (0, 201, -9.0), (0, 640, 30.0), (1, 300, 12.0)]
    c = Case(H + m + K + D, m=[m, m], n=[n, n], H=H, D=D, K=K, columns=n, loud=loud)
    check(c)


@pytest.mark.parametrize("H,m,K", KERNELS)
def test_rows_that_see_nothing(H, m, K):
    """More new tokens than cached positions, no positions, no tokens."""
    sink = torch.randn(H)
    sink[0], sink[1], sink[2] = float("-inf"), float("inf"), 3.0
    c = Case(7, m=[m + 2, m, 0, m], n=[2, 0, 40, 300], H=H, D=512, K=K, sink=sink)
    out, lse = check(c)
    q0 = c.q_indptr_l
    assert bool((out[q0[1]:q0[2]] == 0).all()) and not bool(torch.signbit(out[q0[1]:q0[2]]).any())
    assert torch.equal(lse[q0[1]:q0[2]].cpu(), sink.expand(m, H))
    assert bool((out[q0[3]:, 1] == 0).all())  # a sink of +inf takes all the weight


@pytest.mark.parametrize("H,m,K", KERNELS)
@pytest.mark.parametrize("window,first", [(0, 0), (20, 3)])
def test_values_that_are_not_seen(H, m, K, window, first):
    """Infinities and NaN behind kv_len, in other blocks, before the window and in
    later tokens' rows leave a row as it is."""
    n = [333, 90]
    c = Case(11, m=[m, m], n=n, H=H, D=512, K=K, window=window, first=first)
    rows = [torch_rows(c, b) for b in range(2)]
    used = torch.zeros(c.pool.shape[0], dtype=torch.bool)
    for r in rows:
        used[r] = True
    c.pool[~used.cuda()] = float("nan")
    if window:  # between the first positions and the first token's window
        c.pool[rows[0][first:n[0] - m - window + 1].cuda()] = float("inf")
    if m > 1:
        c.pool[rows[1][-2].cuda(), 5] = float("nan")  # the last token but one, and the last see it
    out, _ = check(c)
    assert bool(torch.isfinite(out[:m]).all())
    if m > 1:
        assert bool(torch.isfinite(out[m:2 * m - 2]).all()) and bool(torch.isnan(out[2 * m - 2:]).all())


def torch_rows(c, b):
    from paged_ref import rows_of
    return rows_of(c.table.cpu().numpy()[b], c.n[b], c.K, c.base)


@pytest.mark.parametrize("H,m,K", KERNELS)
def test_rows_outside_the_sequences_are_left_alone(H, m, K):
    c = Case(3, m=[m, m], n=[100, 30], H=H, D=256, K=K, lead=3, trail=5)
    out = torch.full_like(c.q, 7.0)
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    c.q[:3] = float("nan")
    c.q[-5:] = float("inf")
    check(c, out=out, lse=lse)
    for t in (out, lse):
        assert bool((t[:3] == 7).all()) and bool((t[-5:] == 7).all())


def test_many_sequences_and_many_units():
    """A plan of its own: more than 2048 sequences, more than 4096 units."""
    check(Case(1, m=[1] * 2100, n=[1 + i % 90 for i in range(2100)], H=2, D=64, K=16, columns=40))
    check(Case(2, m=[100] * 41, n=[100 + i for i in range(41)], H=128, D=256, K=16, columns=60))


def test_whole_units_of_a_window():
    """Short spans: units are not cut, with a short table and with a window."""
    check(Case(4, m=[300, 41, 7], n=[900, 41, 500], H=16, D=512, K=16, window=100, first=5))
    check(Case(5, m=[60, 41, 7], n=[300, 41, 200], H=24, D=512, K=16))
    check(Case(6, m=[1] * 5, n=[300, 41, 200, 1, 0], H=24, D=128, K=16))


def test_bad_lengths_and_table_entries():
    c = Case(8, m=[2, 3], n=[100, 200], H=64, D=512, K=16)
    ws = torch.empty(sda.chunk_attention_workspace_size(2, 5, 64, 512), dtype=torch.uint8, device="cuda")
    good, _ = c.attend(sda, workspace=ws)
    assert sda.paged_error_flag(ws) == 0
    out = torch.full_like(c.q, 7.0)
    for name, value in (("kv_len", [100, 100000]), ("kv_len", [-1, 200]), ("q_indptr", [0, 6, 5]),
                        ("q_indptr", [0, 2, 6]), ("q_indptr", [-1, 2, 5])):
        keep = getattr(c, name)
        setattr(c, name, torch.tensor(value, dtype=torch.int32, device="cuda"))
        c.attend(sda, workspace=ws, out=out)
        assert sda.paged_error_flag(ws) == 2
        setattr(c, name, keep)
        assert bool((out == 7).all())
    for entry in (-1, 10 ** 6, 2 ** 31 - 1):
        table = c.table.clone()
        c.table[0, 3] = entry
        got, _ = c.attend(sda, workspace=ws)
        assert sda.paged_error_flag(ws) == 3
        c.table = table
        assert torch.equal(got[2:], good[2:])  # the other sequence's
    c.attend(sda, workspace=ws)
    assert sda.paged_error_flag(ws) == 0


def test_pool_rows_beyond_two_billion_elements():
    base = (1 << 31) // 512 + 1000
    c = Case(9, m=[3, 1], n=[150, 70], H=64, D=512, K=16, device="cpu")
    pool = torch.zeros(base + c.pool.shape[0], 512, dtype=torch.bfloat16, device="cuda")
    pool[base:] = c.pool.cuda()
    ro, rl, to, tl = attend(c)
    c.to("cuda")
    c.pool, c.base = pool, base
    for K in (16, 1):
        if K == 1:
            j = torch.arange(c.table.shape[1] * 16, device="cuda")
            c.table, c.K = (c.table[:, j // 16] * 16 + (j % 16).to(torch.int32)).to(torch.int32), 1
        out, lse = c.attend(sda)
        assert bool(((out.double().cpu() - ro).abs() <= to).all())
        assert bool(((lse.double().cpu() - rl).abs() <= tl).all())


@pytest.mark.parametrize("m,n", [([1, 1, 1], [900, 400, 30]), ([40, 3, 100], [900, 400, 130])])
def test_captured_and_replayed(m, n):
    """A captured call with new contents of its buffers, lengths among them."""
    c = Case(20, m=m, n=n, H=32, D=512, K=64)
    d = Case(21, m=m, n=n, H=32, D=512, K=64)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    ws = torch.empty(sda.chunk_attention_workspace_size(3, c.q.shape[0], 32, 512), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.attend(sda, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(sda, out=out, lse=lse, workspace=ws)
    g.replay()
    first = out.clone()
    want, _ = check(c)
    assert torch.equal(first, want)
    d.n = [x - 7 for x in n]
    d.kv_len = torch.tensor(d.n, dtype=torch.int32, device="cuda")
    want, wl = check(d)
    for name in ("pool", "q", "sink", "table", "kv_len"):
        getattr(c, name).copy_(getattr(d, name))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_two_streams_at_once():
    cases = [Case(30 + i, m=[1 + 60 * i, 5], n=[1500, 700], H=32, D=512, K=16) for i in range(2)]
    want = [c.attend(sda)[0].clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(cases):
            got[i].append(c.attend(sda, stream=streams[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])


def test_one_token_agrees_with_decode():
    """A step's chunk attention and decode() over the same rows' slot lists."""
    from paged_ref import rows_of
    c = Case(40, m=[1, 1, 1], n=[300, 64, 1000], H=64, D=512, K=64)
    lists = [rows_of(c.table.cpu().numpy()[b], c.n[b], c.K, c.base) for b in range(3)]
    idx = torch.cat(lists).to(torch.int32).cuda()
    ptr = torch.tensor([0, 300, 364, 1364], dtype=torch.int32, device="cuda")
    out, _ = check(c)
    ref = sda.decode(c.q, c.pool, idx, ptr, c.sink, c.scale)
    _, _, tol, _ = attend(c)
    assert bool(((out.double() - ref.double()).abs().cpu() <= 2 * tol).all())


@pytest.mark.parametrize("H,m,K", KERNELS)
def test_nan_that_is_seen(H, m, K):
    """A row all of whose positions hold NaN, and one that holds one of them."""
    sink = torch.zeros(H)
    sink[0] = float("-inf")
    c = Case(12, m=[m, m], n=[m, 600], H=H, D=512, K=K, sink=sink, columns=600)
    c.pool[torch_rows(c, 0).cuda()] = float("nan")
    c.pool[torch_rows(c, 1)[500].cuda(), 3] = float("nan")
    out, lse = check(c)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("H,B", [(4, 1), (64, 1), (64, 2049)])
def test_lengths_near_two_billion_are_refused(H, B):
    """Positions are counted in 32 bits, tiles' ends too.  (H = 64, one sequence of 5
    tokens: two CTAs a tile; 2049 sequences: the plan.)"""
    m = 5 if B == 1 else 1
    q = torch.zeros(m * B, H, 512, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(64, 512, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    ptr = torch.arange(0, m * B + 1, m, dtype=torch.int32, device="cuda")
    n = torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    n[1:] = 1
    ws = torch.empty(sda.chunk_attention_workspace_size(B, m * B, H, 512), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    sda.chunk_attention(q, pool, table, ptr, n, torch.zeros(H, device="cuda"), 0.1, k_per_block=2 ** 30, out=out,
                        workspace=ws)
    assert sda.paged_error_flag(ws) == 2
    assert bool((out == 3.0).all())
