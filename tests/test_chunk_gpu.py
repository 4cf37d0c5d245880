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
