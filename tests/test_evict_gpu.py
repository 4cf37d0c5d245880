"""Slot eviction against its definition: exact."""
import numpy as np
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import evict

pytestmark = pytest.mark.gpu


def inputs(seed, B, S, kind="random"):
    rng = np.random.default_rng(seed)
    s = rng.exponential(size=(B, S)).astype(np.float32)
    if kind == "ties":
        s = rng.integers(0, 4, (B, S)).astype(np.float32)
    if kind == "special":
        s = rng.choice(np.array([0.0, -0.0, 1.0, np.inf, -np.inf, np.nan, -1.0, 1e-40], np.float32), (B, S))
    t = rng.permutation(B * S).astype(np.int32).reshape(B, S)
    return torch.from_numpy(s).cuda(), torch.from_numpy(t).cuda()


def same(r, ref, W):
    os, ot, ol, freed, ptr, status = ref
    assert r.kv_len.tolist() == ol
    assert np.array_equal(r.slot_table.cpu().numpy(), ot)
    assert np.array_equal(r.scores.cpu().numpy().view(np.int32), os.view(np.int32))  # bit for bit
    assert r.freed_indptr.tolist() == ptr
    f = r.freed_slots.cpu().numpy()
    assert f[:len(freed)].tolist() == freed and bool((f[len(freed):] == -1).all())
    assert int(r.status.item()) == status


@pytest.mark.parametrize("kind", ["random", "ties", "special"])
@pytest.mark.parametrize("S,budget,first,recent", [
    (1, 1, 0, 0), (1, 0, 0, 0), (7, 3, 1, 1), (64, 63, 0, 63), (100, 100, 0, 0), (700, 512, 4, 128),
    (1025, 1, 0, 0), (1025, 1, 1, 0), (3001, 130, 2, 128), (5000, 4096, 4, 17), (20000, 333, 0, 0),
    (4096, 700, 3, 5), (4097, 700, 3, 5), (210000, 1000, 4, 128)])
def test_evict(kind, S, budget, first, recent):
    B = 5
    s, t = inputs(S + budget, B, S, kind)
    lens = [S, S // 2, 0, min(S, budget), min(S, budget + 1)]
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    W = min(S, budget)
    r = sda.evict_slots(s, t, n, budget, first=first, recent=recent)
    torch.cuda.synchronize()
    ref = evict(s, t, lens, budget, first, recent, W)
    same(r, ref, W)
    # in place: the same numbers, in the inputs' own arrays
    ref = evict(s, t, lens, budget, first, recent, S)
    out = sda.Evicted(s, t, n, r.freed_slots, r.freed_indptr, r.status)
    r = sda.evict_slots(s, t, n, budget, first=first, recent=recent, out=out)
    torch.cuda.synchronize()
    assert r.scores.data_ptr() == s.data_ptr()
    same(r, ref, S)


def test_bad_length_counts_as_zero():
    s, t = inputs(3, 3, 50)
    n = torch.tensor([51, -1, 50], dtype=torch.int32).cuda()
    r = sda.evict_slots(s, t, n, 20)
    torch.cuda.synchronize()
    same(r, evict(s, t, n.tolist(), 20, 0, 0, 20), 20)


@pytest.mark.parametrize("B,S,budget", [(20, 5000, 900), (20, 160000, 4096)])
def test_many_sequences(B, S, budget):
    """More sequences than clusters of 8 that run at once."""
    s, t = inputs(B, B, S)
    lens = np.random.default_rng(B).integers(0, S + 1, B).tolist()
    r = sda.evict_slots(s, t, torch.tensor(lens, dtype=torch.int32).cuda(), budget, first=4, recent=9)
    torch.cuda.synchronize()
    same(r, evict(s, t, lens, budget, 4, 9, budget), budget)


def test_no_sequences():
    """The freed list holds -1 behind its end, also when that is all of it."""
    i32 = dict(dtype=torch.int32, device="cuda")
    out = sda.Evicted(torch.empty(0, 7, device="cuda"), torch.empty(0, 7, **i32), torch.empty(0, **i32),
                      torch.full((5,), 9, **i32), torch.full((1,), 9, **i32), torch.full((1,), 9, **i32))
    r = sda.evict_slots(torch.empty(0, 9, device="cuda"), torch.empty(0, 9, **i32), torch.empty(0, **i32), 7, out=out)
    torch.cuda.synchronize()
    assert r.freed_slots.tolist() == [-1] * 5 and r.freed_indptr.tolist() == [0] and r.status.tolist() == [0]
