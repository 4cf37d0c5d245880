"""Attention mass over a paged cache against its definition in 64 bits."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case, attend, mass

pytestmark = pytest.mark.gpu


def run(c, lse, **kw):
    return sda.attention_mass(c.q, c.pool, c.table, c.q_indptr, c.kv_len, lse, c.scale,
                              k_per_block=c.K, base=c.base, window=c.window, first=c.first, **kw)


def check(c, decay=None):
    lse = attend(c)[1].float().cuda()
    S = c.table.shape[1] * c.K
    prev, kw = None, {}
    if decay is not None:
        prev = torch.rand(c.B, S, generator=torch.Generator().manual_seed(5)).cuda()
        kw = dict(scores=prev, decay=decay)
    got = run(c, lse, **kw)
    torch.cuda.synchronize()
    ref, tol = mass(c, lse, prev, decay if decay is not None else 1.0)
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    assert torch.equal(got, run(c, lse, **kw))  # a fixed order of summation
    return got


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 64, 128])
def test_shapes(D, H):
    check(Case(D + H, m=[1, 3, 0, 7], n=[70, 3, 200, 131], H=H, D=D, K=16))


@pytest.mark.parametrize("K", [1, 3, 16, 64, 100, 128])
def test_block_sizes(K):
    check(Case(K, m=[1, 1, 5, 40], n=[1, 64, 65, 300], H=16, D=512, K=K, base=5), decay=0.5)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 1000, 5000])
def test_one_token(n):
    check(Case(n, m=[1], n=[n], H=16, D=512, K=64), decay=1.0)
    check(Case(n, m=[1] * 3, n=[n, 1, max(1, n // 2)], H=64, D=512, K=1))


@pytest.mark.parametrize("m,n", [([33], [33]), ([64], [640]), ([129], [1000]), ([200, 1, 17], [200, 900, 18])])
def test_chunks(m, n):
    check(Case(sum(n), m=m, n=n, H=8, D=512, K=64))


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (7, 4), (64, 0), (64, 64), (65, 70), (100, 3),
                                          (128, 200), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_window(window, first):
    check(Case(window % 977, m=[1, 90, 13], n=[500, 301, 13], H=16, D=128, K=16, window=window, first=first))
    check(Case(first % 977, m=[40], n=[700], H=16, D=512, K=64, window=window, first=first))


@pytest.mark.parametrize("H,m,K", [(4, 1, 16), (4, 1, 3), (64, 1, 16), (64, 1, 3), (64, 5, 16), (64, 5, 3)])
def test_what_is_not_seen(H, m, K):
    """Garbage behind kv_len and in other sequences' rows stays out; positions behind
    kv_len, and sequences without tokens, get what they should."""
    c = Case(11, m=[m, 0, m, m], n=[333, 50, 90, 0], H=H, D=512, K=K, columns=700 // K, lead=2, trail=3)
    from paged_ref import rows_of
    used = torch.zeros(c.pool.shape[0], dtype=torch.bool)
    for b in range(4):
        used[rows_of(c.table.cpu().numpy()[b], c.n[b], c.K, c.base)] = True
    c.pool[~used.cuda()] = float("nan")
    c.q[:2], c.q[-3:] = float("nan"), float("nan")
    got = check(c, decay=0.25)
    assert bool((got[0, 333:] == 0).all()) and bool((got[3] == 0).all()) and bool((got[1, :50] > 0).any())


def test_in_place_and_without_scores():
    c = Case(12, m=[3, 70], n=[200, 300], H=8, D=256, K=16)
    lse = attend(c)[1].float().cuda()
    S = c.table.shape[1] * 16
    prev = torch.rand(2, S, device="cuda")
    want = run(c, lse, scores=prev, decay=0.75)
    out = run(c, lse, scores=prev, decay=0.75, out=prev)
    assert out.data_ptr() == prev.data_ptr() and torch.equal(out, want)
    assert torch.equal(run(c, lse), run(c, lse, scores=torch.zeros(2, S, device="cuda")))


def test_a_sink_that_takes_all():
    c = Case(13, m=[2], n=[100], H=4, D=64, K=16)
    lse = attend(c)[1].float().cuda()
    lse[:, 1] = float("inf")
    ref, tol = mass(c, lse)
    got = run(c, lse)
    assert bool(((got.double().cpu() - ref).abs() <= tol).all())


def test_weights_sum_to_what_the_sink_leaves():
    """Over a sequence, the weights of each row and its sink's add up to 1."""
    c = Case(14, m=[1, 30], n=[500, 700], H=16, D=512, K=64)
    _, lse = c.attend(sda)
    got = run(c, lse).double().cpu().sum(dim=1)
    left = (1 - torch.exp(c.sink.double()[None] - lse.double())).cpu()
    want = torch.stack([left[:1].sum(), left[1:].sum()])
    # lse and the weights are off by about 2^-20 each, in N = 480 rows at most
    assert bool(((got - want).abs() <= 480 * 2.0 ** -18).all())


def test_bad_lengths_and_table_entries():
    for m in ([1, 1], [200, 3]):
        c = Case(8, m=m, n=[300, 200], H=16, D=512, K=16)
        lse = attend(c)[1].float().cuda()
        ws = torch.empty(sda.attention_mass_workspace_size(2, c.table.shape[1], 16), dtype=torch.uint8,
                         device="cuda")
        S = c.table.shape[1] * 16
        prev = torch.rand(2, S, device="cuda")
        good = run(c, lse, workspace=ws, scores=prev)
        assert sda.paged_error_flag(ws) == 0
        keep = c.kv_len
        c.kv_len = torch.tensor([300, -1], dtype=torch.int32, device="cuda")
        got = run(c, lse, workspace=ws, scores=prev, decay=0.5)
        assert sda.paged_error_flag(ws) == 2
        assert torch.equal(got[0, :300], 0.5 * prev[0, :300]) and bool((got[1] == 0).all())
        c.kv_len = keep
        c.table[0, 3] = 10 ** 6
        got = run(c, lse, workspace=ws, scores=prev)
        assert sda.paged_error_flag(ws) == 3
        assert torch.equal(got[1], good[1]) and torch.equal(got[0, :48], good[0, :48])


def test_captured_and_replayed():
    for m in ([1, 1], [150, 3]):
        c, d = (Case(s, m=m, n=[600, 200], H=16, D=512, K=16) for s in (50, 51))
        l1, l2 = (attend(x)[1].float().cuda() for x in (c, d))
        out = torch.empty(2, c.table.shape[1] * 16, device="cuda")
        ws = torch.empty(sda.attention_mass_workspace_size(2, c.table.shape[1], 16), dtype=torch.uint8,
                         device="cuda")
        run(c, l1, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, l1, out=out, workspace=ws)
        want = run(d, l2)
        for name in ("pool", "q", "table", "kv_len"):
            getattr(c, name).copy_(getattr(d, name))
        l1.copy_(l2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_many_sequences():
    check(Case(15, m=[1] * 2100, n=[1 + i % 90 for i in range(2100)], H=2, D=64, K=16, columns=40))
