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
