"""Head counts, tables and captures that the operators' other tests leave out."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case, evict
from test_chunk_gpu import check
from test_evict_gpu import inputs, same
from test_mass_gpu import check as check_mass

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [128, 129, 200, 255, 256])
@pytest.mark.parametrize("K", [16, 3])
@pytest.mark.parametrize("D", [64, 256, 512])
def test_many_heads_one_token(H, K, D):
    """A step of 128 heads: two units of 64 rows a sequence; of more: pairs where D >= 256."""
    c = Case(H + K + D, m=[1, 1, 1], n=[700, 64, 1], H=H, D=D, K=K)
    check(c)
    check_mass(c, decay=0.5)


@pytest.mark.parametrize("H", [129, 256])
def test_many_heads_chunk(H):
    c = Case(H, m=[5, 0, 33], n=[400, 30, 33], H=H, D=512, K=16, window=70, first=3)
    check(c)
    check_mass(c)


@pytest.mark.parametrize("H,m", [(16, 1), (64, 1), (128, 1), (64, 5)])
@pytest.mark.parametrize("K", [64, 1])
def test_table_far_wider_than_the_sequences(H, m, K):
    c = Case(H + m, m=[m] * 3, n=[300, 64 + m, m], H=H, D=512, K=K, columns=131072 // K)
    check(c)
    got = check_mass(c, decay=1.0)
    for b in range(3):
        assert bool((got[b, c.n[b]:] == 0).all())


def test_skewed_step():
    """All tokens of a step in one sequence: the kernel for steps takes its rows 64 at a time."""
    c = Case(5, m=[0] * 7 + [8] + [0] * 8, n=[40] * 7 + [500] + [3] * 8, H=64, D=512, K=16)
    check(c)
    check_mass(c)


@pytest.mark.parametrize("S", [700, 5000, 210000])
@pytest.mark.parametrize("in_place", [False, True])
def test_captured_eviction(S, in_place):
    """Replayed with other scores, slots and lengths (one CTA, clusters, streamed rows)."""
    B, budget = 3, 500
    W = S if in_place else budget
    i32 = dict(dtype=torch.int32, device="cuda")
    s, t = inputs(1, B, S)
    n = torch.zeros(B, **i32)
    out = sda.Evicted(s if in_place else torch.empty(B, W, device="cuda"), t if in_place else torch.empty(B, W, **i32),
                      n if in_place else torch.empty(B, **i32), torch.empty(B * (S - budget), **i32),
                      torch.empty(B + 1, **i32), torch.empty(1, **i32))
    sda.evict_slots(s, t, n, budget, first=4, recent=100, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sda.evict_slots(s, t, n, budget, first=4, recent=100, out=out)
    for seed, lens in ((2, [S, S // 2, 0]), (3, [501, 500, S]), (4, [S + 1, -1, 499])):
        s2, t2 = inputs(seed, B, S, "special")
        s.copy_(s2)
        t.copy_(t2)
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        same(out, evict(s2, t2, lens, budget, 4, 100, W), W)
