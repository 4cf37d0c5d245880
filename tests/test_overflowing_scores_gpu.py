"""Finite rows whose scores lie below the range of fp32: their weight is 0, wherever they
stand and whatever comes before them."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case, logits, rows_of
from test_chunk_gpu import KERNELS

pytestmark = pytest.mark.gpu

HUGE = 2.0 ** 70  # squared: beyond fp32


@pytest.mark.parametrize("H,m,K", KERNELS + [(4, 30, 16)])
@pytest.mark.parametrize("where", ["first", "all", "last", "some"])
@pytest.mark.parametrize("D", [128, 512])
def test_scores_below_the_range(H, m, K, where, D):
    n = [700, 90]
    c = Case(70 + H + m, m=[m, m], n=n, H=H, D=D, K=K, columns=700)
    c.q[..., 0] = 0
    c.pool[:, 0] = 0
    rows = [rows_of(c.table.cpu().numpy()[b], n[b], K, c.base) for b in range(2)]
    ref = [logits(c, b) for b in range(2)]
    c.q[..., 0] = HUGE
    low = []
    for b in range(2):
        s = torch.zeros(n[b], dtype=torch.bool)
        s[{"first": slice(0, n[b] // 3), "all": slice(0, n[b]), "last": slice(n[b] - m - 20, n[b]),
           "some": slice(1, n[b], 3)}[where]] = True
        c.pool[rows[b][s].cuda(), 0] = -HUGE
        low.append(s)
    out, lse = c.attend(sda)
    got = sda.attention_mass(c.q, c.pool, c.table, c.q_indptr, c.kv_len, lse, c.scale, k_per_block=K)
    out, lse, got, sink = out.double().cpu(), lse.double().cpu(), got.cpu(), c.sink.cpu().double()
    for b in range(2):
        x, kv, _, delta = ref[b]  # of the columns behind the first
        kv[low[b], 0] = -HUGE
        x[..., low[b]] = -float("inf")
        z = torch.logsumexp(torch.cat([x, sink.view(1, H, 1).expand(m, H, 1)], 2), dim=2)
        w = torch.exp(x - z[..., None])
        o, a = torch.einsum("thj,jd->thd", w, kv), torch.einsum("thj,jd->thd", w, kv.abs())
        s = slice(b * m, (b + 1) * m)
        assert bool(((out[s] - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * delta[..., None] + 2.0 ** -18) * a).all())
        assert bool(((lse[s] - z).abs() <= delta + 2.0 ** -20 * (1 + z.abs())).all())
        assert bool((got[b, :n[b]][low[b]] == 0).all())
        if where == "all":
            assert bool((out[s] == 0).all()) and torch.equal(lse[s], sink.expand(m, H))
