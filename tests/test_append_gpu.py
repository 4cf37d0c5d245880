"""The append to a paged cache against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import sink_sda_decode_gb300 as sda
from fp8_ref import E4M3, decode, need_of, rotated
from paged_ref import rows_of

pytestmark = pytest.mark.gpu


class Append:
    """One random call: rows, queries, tables, and a pool with rows in it."""

    def __init__(self, seed, m, n, H=4, D=128, K=16, rope=64, norm=True, fp8=True, base=0, lead=0, trail=0,
                 size=1.0, max_pos=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.m, self.n, self.H, self.D, self.K, self.base, self.fp8 = list(m), list(n), H, D, K, base, fp8
        B = len(m)
        blocks = [-(-max(x, 0) // K) for x in n]
        total = sum(blocks) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((B, max(blocks + [1])), -7, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :blocks[b]] = perm[at:at + blocks[b]]
            at += blocks[b]
        self.ptr = [lead + x for x in np.cumsum([0] + self.m).tolist()]
        T = self.ptr[-1] + trail
        self.kv = (torch.randn(T, D, generator=g) * size).to(torch.bfloat16)
        self.q = torch.randn(T, H, D, generator=g).to(torch.bfloat16) if H else None
        self.kv_w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm else None
        self.q_w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm and H else None
        pos = max(n + [1]) if max_pos is None else max_pos
        ang = torch.arange(pos, dtype=torch.float64)[:, None] * 10000.0 ** -(torch.arange(rope // 2) / max(rope // 2, 1))
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        rows = base + total * K
        if fp8:
            self.pool = torch.randint(0, 127, (rows, D), generator=g, dtype=torch.uint8)
            self.pool += 128 * torch.randint(0, 2, (rows, D), generator=g, dtype=torch.uint8)
            self.scale = torch.exp2(torch.randint(-9, -4, (total,), generator=g).float())
        else:
            self.pool = torch.randn(rows, D, generator=g).to(torch.bfloat16)
            self.scale = None

    def cuda(self):
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.d = {k: up(getattr(self, k)) for k in ("kv", "q", "kv_w", "q_w", "cos", "sin", "table", "pool", "scale")}
        self.d["ptr"] = torch.tensor(self.ptr, dtype=torch.int32, device="cuda")
        self.d["n"] = torch.tensor(self.n, dtype=torch.int32, device="cuda")
        return self

    def call(self, **kw):
        d = self.d
        pool = {"kv_fp8": d["pool"], "block_scale": d["scale"]} if self.fp8 else {"unified_kv": d["pool"]}
        return sda.append_rows(d["kv"], d["cos"], d["sin"], d["table"], d["ptr"], d["n"], k_per_block=self.K,
                               base=self.base, kv_norm_w=d["kv_w"], q=d["q"], q_norm_w=d["q_w"], eps=1e-6,
                               **pool, **kw)


def check(a, status=0, skip=(), **kw):
    """One call; every output, and every row and scale that has to stay as it was."""
    if not hasattr(a, "d"):
        a.cuda()
    q_out, st = a.call(**kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    pool, scale = a.d["pool"].cpu(), None if a.scale is None else a.d["scale"].cpu()
    touched, blocks = torch.zeros(pool.shape[0], dtype=torch.bool), set()
    max_pos = a.cos.shape[0] if a.cos.shape[1] else 2 ** 31
    for b in range(len(a.m)):
        if b in skip or a.m[b] == 0:
            continue
        pos = torch.arange(a.n[b] - a.m[b], a.n[b])
        ok = (pos >= 0) & (pos < max_pos)
        t = torch.arange(a.ptr[b], a.ptr[b + 1])
        if a.H:
            y, tol = rotated(a.q[t[ok]], a.q_w, 1e-6, pos[ok], a.cos, a.sin)
            got = q_out[t].double().cpu()
            assert bool(((got[ok] - y).abs() <= 2.0 ** -8 * y.abs() + 1.01 * tol).all())
            assert bool((got[~ok] == 0).all())
        if not bool(ok.any()):
            continue
        pos, t = pos[ok], t[ok]
        y, tol = rotated(a.kv[t], a.kv_w, 1e-6, pos, a.cos, a.sin)
        row = rows_of(a.table.numpy()[b], int(pos[-1]) + 1, a.K, a.base)[pos]
        if not a.fp8:
            touched[row] = True
            assert bool(((pool[row].double() - y).abs() <= 2.0 ** -8 * y.abs() + 1.01 * tol).all())
            continue
        for j in sorted(set((pos // a.K).tolist())):
            mine = pos // a.K == j
            blk = int(a.table[b, j])
            blocks.add(blk)
            finite = torch.isfinite(y[mine])
            top = torch.where(finite, y[mine].abs(), torch.zeros_like(y[mine]))
            err = float(torch.where(finite, tol[mine], torch.zeros_like(top)).max())
            can = {need_of(max(float(top.max()) + e, 0.0)) for e in (-err, err)}
            held = int(pos[mine][0]) % a.K
            s = float(scale[blk])
            old = float(a.scale[blk])
            assert s in ({max(c, old) for c in can} if held else can), (s, can, old, held)
            first = a.base + blk * a.K
            if held:
                was, now = a.pool[first:first + held], pool[first:first + held]
                if s == old:
                    assert torch.equal(was, now)
                else:
                    v = decode(was) * old
                    assert torch.equal(torch.isnan(v), torch.isnan(decode(now)))
                    off = (decode(now) * s - v).abs()
                    # (the factor old / new is rounded to fp32, and the product)
                    lim = torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10)) * (1 + 2.0 ** -20)
                    assert bool((off <= lim)[~torch.isnan(v)].all())
                touched[first:first + held] = True
            touched[row[mine]] = True
            got = decode(pool[row[mine]]) * s
            assert torch.equal(torch.isnan(got), ~finite)
            lim = torch.maximum(y[mine].abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10)) + 1.1 * tol[mine]
            assert bool(((got - y[mine]).abs() <= lim)[finite].all())
    assert torch.equal(pool[~touched], a.pool[~touched])
    if a.fp8:
        same = torch.tensor([x not in blocks for x in range(a.scale.numel())])
        assert torch.equal(scale[same], a.scale[same])
    return q_out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,rope", [(16, 0), (16, 16), (64, 32), (128, 128), (256, 64), (512, 64), (528, 64),
                                    (1024, 1024), (192, 8)])
def test_widths(D, rope, fp8):
    check(Append(D + rope, m=[1, 20, 0, 7], n=[5, 33, 9, 7], D=D, rope=rope, fp8=fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("H", [0, 1, 5, 64])
def test_heads(H, norm, fp8):
    check(Append(H, m=[1, 3, 40], n=[70, 3, 131], H=H, D=512, K=64, norm=norm, fp8=fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K", [1, 2, 3, 16, 64, 100, 1000])
def test_block_sizes(K, fp8):
    a = Append(K, m=[1, 1, 5, 40, 300], n=[1, K, K + 1, 2 * K + 40, 300 + K // 2], K=K, fp8=fp8, base=5)
    check(a, status=int(K + 1 < 5))  # (five tokens then have fewer positions)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [1, 2, 127, 128, 129, 700, 17000])
def test_many_sequences(B, fp8):
    """The search for a token's sequence in one, two and three steps; empty sequences."""
    m = [(i * 7) % 3 for i in range(B)]
    m[-1] = 1
    check(Append(B, m=m, n=[x + (i * 5) % 11 for i, x in enumerate(m)], H=1, D=64, K=4, rope=8, fp8=fp8))


@pytest.mark.parametrize("K", [16, 64])
@pytest.mark.parametrize("size", [1e-3, 0.05, 1.0, 300.0, 1e30])
def test_scales_that_grow_and_stay(K, size):
    """Blocks with rows in them: codes that stay, and codes that are rounded again."""
    check(Append(3, m=[1, 5, 30, 70], n=[K + 3, 10, 41, 200], H=0, K=K, norm=False, size=size))
    a = Append(4, m=[2, 3], n=[20, 9], H=0, K=K, norm=False, size=size)
    a.scale = torch.rand(a.scale.numel(), generator=torch.Generator().manual_seed(1)) / 50  # not powers of two
    a.scale[int(a.table[0, 0])] = 0.0
    check(a)


def test_exact_powers():
    """Largest elements of exactly 448 * 2^e need 2^e, the next value the next power."""
    for top, want in ((448.0, 1.0), (450.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7), (0.0, 2.0 ** -126),
                      (2.0 ** -133, 2.0 ** -126)):
        a = Append(5, m=[3], n=[3], H=0, K=4, rope=0, norm=False)
        a.kv = torch.zeros_like(a.kv)
        a.kv[1, 9] = -top
        check(a)
        assert float(a.d["scale"][int(a.table[0, 0])]) == want
    # rows after a block of zeros set the scale as if they were first
    a = Append(6, m=[2], n=[2], H=0, K=8, rope=0, norm=False)
    a.kv = torch.zeros_like(a.kv)
    check(a)
    b = Append(7, m=[1], n=[3], H=0, K=8, rope=0, norm=False, size=0.01)
    b.table, b.scale, b.pool = a.table, a.d["scale"].cpu(), a.d["pool"].cpu()
    check(b)


def test_values_that_are_not_finite():
    """Infinities and NaN become NaN codes and leave their block's scale alone."""
    a = Append(8, m=[4, 2], n=[6, 2], H=2, K=4, norm=False, rope=0)
    a.kv[0, 3], a.kv[1, 5], a.kv[4, 0] = float("inf"), float("nan"), float("-inf")
    check(a)
    b = Append(8, m=[4], n=[6], H=0, K=4, norm=True)
    b.kv[2, 7] = float("nan")  # its whole row
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_positions_outside(fp8):
    """More tokens than positions, and positions behind the rotation's caches."""
    a = Append(9, m=[7, 5, 3], n=[4, 60, 3], fp8=fp8, max_pos=57)
    check(a, status=1)
    check(Append(10, m=[7, 5], n=[0, 60], fp8=fp8, rope=0, max_pos=0), status=1)
    check(Append(10, m=[7, 5], n=[7, 60], fp8=fp8, rope=0, max_pos=0))
    check(Append(11, m=[3], n=[3], fp8=fp8, max_pos=0), status=1)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_outside_the_sequences_are_left_alone(fp8):
    a = Append(12, m=[2, 3], n=[9, 40], lead=3, trail=4, fp8=fp8).cuda()
    out = torch.full_like(a.d["q"], 7.0)
    check(a, q_out=out)
    assert bool((out[:3] == 7).all()) and bool((out[-4:] == 7).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_table_entries(fp8):
    good = dict(m=[2, 3, 4], n=[20, 30, 40])
    for field, value, skip in (("n", [20, 10 ** 6, 40], (1,)), ("n", [-1, 30, 40], (0,)), ("n", [2 ** 31 - 1, 30, 40], (0,))):
        a = Append(13, **good, fp8=fp8).cuda()
        a.d["n"] = torch.tensor(value, dtype=torch.int32, device="cuda")
        out = torch.full_like(a.d["q"], 7.0)
        check(a, status=4, skip=skip, q_out=out)
        for b in skip:
            assert bool((out[a.ptr[b]:a.ptr[b + 1]] == 7).all())
    for ptr in ([0, 2, 1, 9], [0, 2, 5, 10], [-1, 2, 5, 9], [9, 0, 0, 0], [0, 2 ** 31 - 1, 5, 9]):
        a = Append(13, **good, fp8=fp8).cuda()
        a.d["ptr"] = torch.tensor(ptr, dtype=torch.int32, device="cuda")
        _, st = a.call()
        assert int(st.item()) & 4
    a = Append(13, m=[0, 2], n=[10 ** 6, 5], fp8=fp8)
    a.n[0] = 3
    a.cuda()
    a.d["n"] = torch.tensor([10 ** 6 + 1, 5], dtype=torch.int32, device="cuda")  # (the table holds 10 ** 6)
    check(a, status=4)  # a sequence without tokens is looked at, too
    for entry in (-1, 10 ** 6, 2 ** 31 - 1):
        a = Append(14, **good, fp8=fp8).cuda()
        a.d["table"][1, 29 // 16] = entry
        before = a.pool.clone()
        _, st = a.call()
        assert int(st.item()) == 2
        rows = rows_of(a.table.numpy()[1], 30, 16, 0)[27:]
        assert torch.equal(a.d["pool"].cpu()[rows], before[rows])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,m,K", [(1, 700, 16), (3, 40, 16), (200, 2, 16), (256, 1, 1), (257, 1, 1), (300, 40, 16),
                                   (2, 600, 1)])
def test_status_word(B, m, K, fp8):
    """Each of its bits, from the first and the last sequence, block and token."""
    a = Append(60 + B, m=[m] * B, n=[m + 5] * B, H=1, D=64, K=K, rope=32, fp8=fp8).cuda()
    table, n, ptr = a.d["table"], a.d["n"], a.d["ptr"]

    def status():
        st = a.call()[1]
        return int(st.item())

    assert status() == 0
    first, last = 5 // K, (m + 4) // K  # blocks that are written
    for b in {0, B // 2, B - 1}:
        for j in {first, (first + last) // 2, last}:
            for entry in (-1, 10 ** 6, 2 ** 31 - 1):
                a.d["table"] = table.clone()
                a.d["table"][b, j] = entry
                assert status() == 2
        a.d["table"] = table
        a.d["n"] = n.clone()
        for length, word in ((m - 1, 1), (-1, 4), (10 ** 9, 4)):
            a.d["n"][b] = length
            assert status() == word
        a.d["n"] = n
    a.d["ptr"] = ptr.clone()
    a.d["ptr"][B] += 1
    assert status() == 4
    a.d["ptr"] = ptr
    if first > 0:  # a block that is not written
        a.d["table"] = table.clone()
        a.d["table"][0, 0] = -1
        assert status() == 0
    a.d["table"] = table
    a.d["n"] = n.clone()
    a.d["n"][B - 1] = m - 1
    a.d["table"] = table.clone()
    a.d["table"][0, last] = -5
    if B > 1:
        assert status() == 3


@pytest.mark.parametrize("fp8", [False, True])
def test_a_pool_that_ends_inside_a_block(fp8):
    a = Append(15, m=[20], n=[20], H=0, K=16, fp8=fp8, spare=0)
    last = int(a.table[0].argmax())  # the pool's last block holds positions 16 last ..
    a.pool = a.pool[:16 + 2].clone()
    a.cuda()
    _, st = a.call()
    pos = 16 * last + torch.arange(16)
    assert int(st.item()) == (2 if int((pos < 20).sum()) > 2 else 0)


def test_in_place_and_given_outputs():
    a = Append(16, m=[3, 9], n=[30, 9], H=16, D=512).cuda()
    want, _ = a.call()
    st = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    q = a.d["q"]
    got, s2 = a.call(q_out=q, status=st)
    assert got is q and s2 is st and int(st.item()) == 0 and torch.equal(q, want)


def test_float8_tensor_is_taken():
    a, b = Append(17, m=[3], n=[30], H=0).cuda(), Append(17, m=[3], n=[30], H=0).cuda()
    a.call()
    b.d["pool"] = b.d["pool"].view(E4M3)
    b.call()
    assert torch.equal(a.d["pool"], b.d["pool"].view(torch.uint8)) and torch.equal(a.d["scale"], b.d["scale"])


@pytest.mark.parametrize("fp8", [False, True])
def test_pool_rows_beyond_two_billion_elements(fp8):
    base = (1 << 32) // 512 + 1000 if fp8 else (1 << 31) // 512 + 1000
    a = Append(18, m=[3, 40], n=[20, 40], H=1, D=512, fp8=fp8).cuda()
    a.call()
    b = Append(18, m=[3, 40], n=[20, 40], H=1, D=512, fp8=fp8).cuda()
    pool = torch.zeros(base + b.pool.shape[0], 512, dtype=b.pool.dtype, device="cuda")
    pool[base:] = b.d["pool"]
    b.d["pool"], b.base = pool, base
    b.call()
    assert torch.equal(pool[base:], a.d["pool"]) and not bool(pool[:base].any())


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed(fp8):
    """A captured call with other contents of its buffers, lengths among them."""
    a = Append(19, m=[1, 4], n=[17, 40], H=8, D=512, fp8=fp8).cuda()
    out, st = torch.empty_like(a.d["q"]), torch.empty(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.call(q_out=out, status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(q_out=out, status=st)
    b = Append(20, m=[1, 4], n=[18, 37], H=8, D=512, fp8=fp8)
    for k in ("kv", "q", "kv_w", "q_w", "table", "pool", "scale"):
        if getattr(b, k) is not None:
            src = getattr(b, k)
            a.d[k].copy_(src)
    a.d["n"].copy_(torch.tensor(b.n, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    b.cuda()
    b.d["cos"], b.d["sin"] = a.d["cos"], a.d["sin"]
    want, ws = b.call()
    assert torch.equal(out, want) and torch.equal(st, ws)
    assert torch.equal(a.d["pool"], b.d["pool"])


def test_on_another_stream():
    a, b = Append(21, m=[3, 90], n=[30, 90], H=16, D=512).cuda(), Append(21, m=[3, 90], n=[30, 90], H=16, D=512).cuda()
    want, _ = a.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, st = b.call(stream=s)
    s.synchronize()
    assert torch.equal(got, want) and int(st.item()) == 0 and torch.equal(a.d["pool"], b.d["pool"])


def test_nothing_to_do():
    a = Append(22, m=[0, 0], n=[3, 0], H=2).cuda()
    before = a.d["pool"].clone()
    q, st = a.call()
    assert q.shape[0] == 0 and int(st.item()) == 0 and torch.equal(a.d["pool"], before)


def test_step_by_step_is_the_cache_that_attention_reads():
    """Prompt, then steps, appended and attended over: against attention in 64 bits over
    the rows as they were appended, within the roundings of both."""
    from fp8_ref import Case8, check8
    D, K, H, steps = 512, 16, 16, 5
    m0, n0 = [30, 50], [30, 50]
    g = torch.Generator().manual_seed(23)
    c = Case8(23, m=[1, 1], n=[x + steps for x in n0], H=H, D=D, K=K)
    codes, scales = c.codes.view(torch.uint8), c.scales
    cos = torch.cos(torch.rand(64, 32, generator=g) * 6).cuda()
    sin = torch.sin(torch.rand(64, 32, generator=g) * 6).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    call = dict(k_per_block=K, kv_norm_w=w, q_norm_w=w, kv_fp8=codes, block_scale=scales)
    for step in range(steps + 1):
        m = m0 if step == 0 else [1, 1]
        n = [x + step for x in n0]
        T = sum(m)
        kv = torch.randn(T, D, generator=g).to(torch.bfloat16).cuda()
        q = torch.randn(T, H, D, generator=g).to(torch.bfloat16).cuda()
        ptr = torch.tensor([0, m[0], T], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(n, dtype=torch.int32, device="cuda")
        q, st = sda.append_rows(kv, cos, sin, c.table, ptr, kv_len, q=q, **call)
        assert int(st.item()) == 0
        c.q, c.q_indptr, c.q_indptr_l, c.kv_len, c.n, c.m = q, ptr, [0, m[0], T], kv_len, n, m
        c.of = scales.cpu().double()[torch.arange(codes.shape[0]) // K]
        c.worth()
        check8(sda, c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,rope", [(16, 16), (64, 32), (128, 64), (192, 8), (256, 256), (512, 64), (528, 64), (1024, 1024)])
def test_same_bits_as_the_ring_store(D, rope, fp8):
    """A row is the same in both stores (a block of one row has the ring's scale)."""
    T = 300
    a = Append(70 + D, m=[T], n=[T], H=5, D=D, K=1, rope=rope, fp8=fp8).cuda()
    q, _ = a.call()
    d = a.d
    ring = torch.zeros(T, D, dtype=d["pool"].dtype, device="cuda")
    scale = torch.zeros(T, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    q2, _ = sda.qk_norm_rope_swa_store(d["q"], d["kv"], d["q_w"], d["kv_w"], d["cos"], d["sin"], pos,
                                       torch.zeros_like(pos), eps=1e-6, win=T, swa_pages=T,
                                       **(dict(kv_fp8=ring, kv_scale=scale) if fp8 else dict(unified_kv=ring)))
    rows = d["table"][0, :T].long()
    assert torch.equal(q.view(torch.int16), q2.view(torch.int16))
    assert torch.equal(d["pool"][rows], ring)
    if fp8:
        assert torch.equal(d["scale"][rows], scale)


def same_cache(a, b):
    return torch.equal(a["pool"], b["pool"]) and torch.equal(a["scale"], b["scale"])


def test_scales_of_a_captured_call():
    """A replay with other rows, lengths and scales writes the scales, too."""
    a = Append(24, m=[1, 4, 40], n=[32, 48, 96], H=2, D=512).cuda()
    out, st = torch.empty_like(a.d["q"]), torch.empty(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.call(q_out=out, status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(q_out=out, status=st)
    for seed, n, size in ((25, [18, 37, 81], 0.01), (26, [17, 40, 90], 50.0)):
        b = Append(seed, m=[1, 4, 40], n=n, H=2, D=512, size=size, norm=False)
        b.kv_w, b.q_w = a.kv_w, a.q_w
        for k in ("kv", "q", "pool", "scale"):
            a.d[k].copy_(getattr(b, k))
        a.d["table"].fill_(-7)
        a.d["table"][:, :b.table.shape[1]] = b.table.cuda()
        a.d["n"].copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        b.cuda()
        b.d["cos"], b.d["sin"] = a.d["cos"], a.d["sin"]
        want, ws = b.call()
        assert torch.equal(out, want) and int(st.item()) == int(ws.item()) == 0
        assert same_cache(a.d, b.d) and not torch.equal(b.d["scale"].cpu(), b.scale)


def test_scales_on_another_stream_and_at_a_large_base():
    a, b, c = (Append(27, m=[3, 40], n=[20, 70], H=1, D=512).cuda() for _ in range(3))
    a.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b.call(stream=s)
    s.synchronize()
    assert same_cache(a.d, b.d)
    base = (1 << 32) // 512 + 1000
    pool = torch.zeros(base + c.pool.shape[0], 512, dtype=torch.uint8, device="cuda")
    pool[base:] = c.d["pool"]
    c.d["pool"], c.base = pool, base
    c.call()
    assert torch.equal(pool[base:], a.d["pool"]) and torch.equal(c.d["scale"], a.d["scale"])
    assert not torch.equal(a.d["scale"].cpu(), a.scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_without_queries_of_many_tokens(fp8):
    """A warp's rows are then of one token each."""
    check(Append(28, m=[5000, 0, 3, 4100], n=[5000, 9, 300, 4500], H=0, D=64, K=16, rope=32, fp8=fp8, trail=7))
    check(Append(29, m=[1000, 1000], n=[1500, 1000], H=3, D=64, K=16, rope=32, fp8=fp8, lead=5))


def test_refusals_say_what_is_wrong():
    for rope, D in ((4, 64), (20, 64), (72, 64)):
        a = Append(30, m=[2], n=[9], H=0, D=D, rope=rope).cuda()
        before = a.d["pool"].clone()
        with pytest.raises(ValueError, match="multiple of 4 columns"):
            a.call()
        assert torch.equal(a.d["pool"], before)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ptr", [[0, 100, 3, 5], [0, 4, 3, 3], [0, 3, 2, 5]])
def test_descending_bounds_touch_nothing_else(ptr, fp8):
    """Sequences beside a bad one are stored or left out; the rest of the pool stays."""
    a = Append(31, m=[3, 1, 1], n=[20, 30, 40], H=2, fp8=fp8).cuda()
    a.d["ptr"] = torch.tensor(ptr, dtype=torch.int32, device="cuda")
    _, st = a.call()
    assert int(st.item()) == 4
    may = torch.zeros(a.pool.shape[0], dtype=torch.bool)
    for b in range(3):
        if 0 <= ptr[b] <= ptr[b + 1] <= 5:
            n = a.n[b]
            blocks = range((n - (ptr[b + 1] - ptr[b])) // a.K, -(-n // a.K))  # (codes of a block may be rounded again)
            for j in blocks:
                first = int(a.table[b, j]) * a.K
                may[first:first + a.K] = True
    assert torch.equal(a.d["pool"].cpu()[~may], a.pool[~may])


def replayed(f, n=10):
    torch.cuda.synchronize()  # (the other stream comes after this one's work)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            f()
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("live", [[0], [0, 1, 700, 4095], [4095], [5, 6]])
def test_padded_batch(live, fp8):
    """4096 sequences of which a few have a token, and rows for all: right, and no slower than the
    full batch by more than a factor (one by one, empty sequences took 27 times as long)."""
    B = 4096
    m = [int(b in live) for b in range(B)]
    a = Append(32, m=m, n=[3 + x for x in m], H=2, D=64, K=4, rope=8, fp8=fp8, trail=B - len(live))
    check(a)
    out, st = torch.empty_like(a.d["q"]), torch.empty(1, dtype=torch.int32, device="cuda")
    padded = replayed(lambda: a.call(q_out=out, status=st))
    a.d["ptr"] = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    full = replayed(lambda: a.call(q_out=out, status=st))
    assert padded < 3 * full + 20, (padded, full)


@pytest.mark.parametrize("fp8", [False, True])
def test_runs_of_empty_sequences(fp8):
    """Of one and of many, in front, between and behind, beside bad ones."""
    m = [0] * 300 + [3] + [0] + [2, 1] + [0] * 129 + [40, 0, 0, 1] + [0] * 200 + [5] + [0] * 50
    check(Append(33, m=m, n=[x + i % 9 for i, x in enumerate(m)], H=3, D=64, K=4, rope=8, fp8=fp8, lead=2, trail=9))
    a = Append(34, m=m, n=[x + i % 9 for i, x in enumerate(m)], H=3, D=64, K=4, rope=8, fp8=fp8).cuda()
    bad = [299, 301, 310, 311, 433, 434, len(m) - 1]
    a.d["n"][bad] = -1
    check(a, status=4, skip=bad)
