"""Blocks that lie partly behind the pool's end, on pools that hold whole groups of 8 rows
(cached rows in boxes of 16) and that do not (row by row): the error word is 3 if a position
there is seen, and 0 if not."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case, attend
from test_chunk_gpu import check

pytestmark = pytest.mark.gpu


def case(H, m, K, cut, n0, window=0, first=0):
    """Two sequences; the first one's last block is the pool's last, `cut` rows of which are missing."""
    c = Case(H + m + K, m=[m, m], n=[n0, 320], H=H, D=512, K=K, base=5, spare=0, window=window, first=first)
    blocks = -(-n0 // K)
    top = int(c.table[c.table >= 0].max())
    b, i = [int(x) for x in (c.table == top).nonzero()[0]]
    c.table[b, i] = c.table[0, blocks - 1].clone()
    c.table[0, blocks - 1] = top
    c.pool = c.pool[:-cut].contiguous()
    return c


def words(c):
    """Error words of the attention and of the mass, and the second sequence's out and mass."""
    B, T, H = 2, c.q.shape[0], c.q.shape[1]
    w1 = torch.empty(sda.chunk_attention_workspace_size(B, T, H, 512), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(sda.attention_mass_workspace_size(B, c.table.shape[1], c.K), dtype=torch.uint8, device="cuda")
    out, lse = c.attend(sda, workspace=w1)
    got = sda.attention_mass(c.q, c.pool, c.table, c.q_indptr, c.kv_len, lse, c.scale, k_per_block=c.K, base=c.base,
                             window=c.window, first=c.first, workspace=w2)
    return sda.paged_error_flag(w1), sda.paged_error_flag(w2), out[c.q_indptr_l[1]:], got[1]


@pytest.mark.parametrize("cut", [8, 24, 5])
@pytest.mark.parametrize("H,m", [(4, 1), (64, 1), (64, 5)])
@pytest.mark.parametrize("K", [16, 64])
def test_block_that_ends_behind_the_pool(H, m, K, cut):
    if cut >= K:
        cut -= 16
    n = 320  # whole blocks: the missing rows are seen
    c = case(H, m, K, cut, n)
    a, b, out, mass = words(c)
    assert (a, b) == (3, 3)
    c.pool = torch.cat([c.pool, torch.ones(cut, 512, dtype=torch.bfloat16, device="cuda")])
    a, b, _, mass_w = words(c)
    assert (a, b) == (0, 0)
    # the other sequence's: its lse, of a size below 15, is off by up to 2^-20 of 1 + |lse| in either call
    ro, _, tol, _ = attend(c)
    assert bool(((out.double().cpu() - ro[m:]).abs() <= tol[m:]).all())
    assert torch.allclose(mass, mass_w, rtol=2 * 16 * 2.0 ** -20, atol=1e-6)
    # the last `cut` positions do not exist: nothing behind the pool is seen
    c = case(H, m, K, cut, n - cut)
    check(c)
    assert words(c)[:2] == (0, 0)


@pytest.mark.parametrize("H,m", [(4, 1), (64, 1), (64, 5)])
@pytest.mark.parametrize("first,word", [(0, 0), (8, 0), (9, 3), (16, 3)])
def test_first_positions_and_a_window(H, m, first, word):
    """The box that straddles the pool's end is the sequence's first; its second half is behind
    the window, and seen only as first positions."""
    c = Case(3, m=[m, m], n=[320, 100], H=H, D=512, K=16, base=5, spare=0, window=30, first=first)
    top = int(c.table[c.table >= 0].max())
    b, i = [int(x) for x in (c.table == top).nonzero()[0]]
    c.table[b, i] = c.table[0, 0].clone()
    c.table[0, 0] = top
    c.pool = c.pool[:-8].contiguous()
    assert words(c)[0] == word
