"""The paged-cache operators in 64 bits, row by row, and the inputs of their tests.

Tolerances (derived, per element): a bf16 result is off by at most half a step,
2^-8 of itself; a weight rounded to bf16 by 2^-8 of itself, which moves a
weighted sum of v by at most 2^-8 * sum_j w_j |v_j|; an fp32 logit summed over D
products by at most delta = D * 2^-23 * scale * sum_d |q_d k_d| (one rounding or
truncation per addition), which moves a weight and the denominator by that share
each; the hardware's 2^x and log2 by about 2^-21.
"""
from __future__ import annotations

import numpy as np
import torch


def rows_of(table_row, n, K, base):
    j = np.arange(n)
    return torch.from_numpy(base + table_row[j // K].astype(np.int64) * K + j % K)


def visible(m, n, window, first):
    """[m, n] bool: which positions each new token sees."""
    p = np.arange(n - m, n)[:, None]
    j = np.arange(n)[None]
    see = j <= p
    if window:
        see = see & ((j > p - window) | (j < first))
    return torch.from_numpy(see)


def logits(c, b):
    """(x [m, H, n] scaled logits, masked -inf; kv [n, D]; delta [m, H]) of sequence b."""
    q = c.q.cpu().double()[c.q_indptr_l[b]:c.q_indptr_l[b + 1]]
    m, n = q.shape[0], c.n[b]
    kv = c.pool.cpu().double()[rows_of(c.table.cpu().numpy()[b], n, c.K, c.base)]
    see = visible(m, n, c.window, c.first)[:, None]
    x = torch.einsum("thd,jd->thj", q, kv) * c.scale
    x = torch.where(see, x, torch.full_like(x, -float("inf")))
    size = torch.einsum("thd,jd->thj", q.abs(), kv.abs()) * abs(c.scale)
    size = torch.where(see, size, torch.zeros_like(size))
    delta = size.amax(dim=2) if n else torch.zeros(m, q.shape[1], dtype=torch.float64)
    return x, kv, see, delta * q.shape[2] * 2.0 ** -23


def attend(c):
    """out [T, H, D], lse [T, H], and how far each may be off."""
    T, H, D = c.q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.zeros(T, H, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    sink = c.sink.cpu().double()
    for b in range(c.B):
        s = slice(c.q_indptr_l[b], c.q_indptr_l[b + 1])
        if s.stop == s.start:
            continue
        x, kv, see, delta = logits(c, b)
        z = torch.logsumexp(torch.cat([x, sink.view(1, H, 1).expand(x.shape[0], H, 1)], 2), dim=2)
        zs = torch.where(torch.isinf(z), torch.zeros_like(z), z)
        w = torch.where(torch.isinf(z)[..., None], torch.zeros_like(x), torch.exp(x - zs[..., None]))
        # a position that a row does not see takes no part, whatever its row holds
        o = torch.einsum("thj,jd->thd", w, torch.nan_to_num(kv, nan=0.0, posinf=0.0, neginf=0.0))
        bad = ~torch.isfinite(kv).all(dim=1)
        hit = (see[:, 0] & bad[None]).any(dim=1)
        o[hit] = float("nan")
        z[hit] = float("nan")
        out[s], lse[s] = o, z
        a = torch.einsum("thj,jd->thd", w, torch.nan_to_num(kv, nan=0.0, posinf=0.0, neginf=0.0).abs())
        tol_o[s] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * delta[..., None] + 2.0 ** -18) * a
        tol_l[s] = delta + 2.0 ** -20 * (1 + torch.where(torch.isfinite(z), z.abs(), torch.zeros_like(z)))
    return out, lse, tol_o, tol_l


class Case:
    """One random input: pool, block table (distinct blocks in random order), q."""

    def __init__(self, seed, m, n, H, D, K, window=0, first=0, base=0, spare=2, device="cuda",
                 scale=None, lead=0, trail=0, sink=None, columns=0, loud=()):
        g = torch.Generator().manual_seed(seed)
        self.m, self.n, self.K, self.base = list(m), list(n), K, base
        self.B, self.window, self.first = len(m), window, first
        self.scale = scale if scale is not None else D ** -0.5
        blocks = [-(-x // K) for x in n]
        mb = max(blocks + [1, columns])
        total = sum(blocks) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.full((self.B, mb), -7, dtype=torch.int32)  # never read behind kv_len
        at = 0
        for b in range(self.B):
            table[b, :blocks[b]] = perm[at:at + blocks[b]]
            at += blocks[b]
        self.pool = torch.randn(base + total * K, D, generator=g).to(torch.bfloat16)
        for b, j, factor in loud:  # rows whose scores stand out
            self.pool[rows_of(table.numpy()[b], n[b], K, base)[j]] *= factor
        self.q_indptr_l = [lead + x for x in np.cumsum([0] + list(m)).tolist()]
        T = self.q_indptr_l[-1] + trail
        self.q = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
        self.sink = torch.randn(H, generator=g) if sink is None else sink
        self.table = table
        self.kv_len = torch.tensor(self.n, dtype=torch.int32)
        self.q_indptr = torch.tensor(self.q_indptr_l, dtype=torch.int32)
        self.to(device)

    def to(self, device):
        for k in ("pool", "q", "sink", "table", "kv_len", "q_indptr"):
            setattr(self, k, getattr(self, k).to(device))
        return self

    def attend(self, sda, **kw):
        return sda.chunk_attention(self.q, self.pool, self.table, self.q_indptr, self.kv_len,
                                   self.sink, self.scale, k_per_block=self.K, base=self.base,
                                   window=self.window, first=self.first, **kw)


def mass(c, lse, prev=None, decay=1.0):
    """out [B, S] and how far each entry may be off.  An fp32 sum of N terms in a
    fixed order, in groups, is off by at most (N + 2) * 2^-24 of the sum of sizes."""
    S = c.table.shape[1] * c.K
    out = torch.zeros(c.B, S, dtype=torch.float64)
    if prev is not None:
        out += decay * prev.cpu().double()
    for b in range(c.B):
        out[b, c.n[b]:] = 0
    tol = out.abs() * 2.0 ** -22
    for b in range(c.B):
        s = slice(c.q_indptr_l[b], c.q_indptr_l[b + 1])
        if s.stop == s.start or c.n[b] == 0:
            continue
        x, _, see, delta = logits(c, b)
        z = lse.cpu().double()[s][..., None]
        w = torch.where(see & (z != float("inf")), torch.exp(x - z), torch.zeros_like(x))
        N = x.shape[0] * x.shape[1]
        out[b, :c.n[b]] += w.sum(dim=(0, 1))
        # the argument of 2^x is rounded to 2^-24 of its size, its result to about 2^-21
        arg = torch.where(see, x.abs() + z.abs(), torch.zeros_like(x)).nan_to_num(posinf=0.0)
        rel = delta[..., None] + arg * 2.0 ** -22 + 2.0 ** -21 + (N + 2) * 2.0 ** -24
        tol[b, :c.n[b]] += torch.where(w > 0, w * rel, w).sum(dim=(0, 1)) + 2.0 ** -120 * N
    return out, tol


def evict(scores, slots, lens, budget, first, recent, W):
    """The definition, sequence by sequence, with Python's own sort."""
    B, S = scores.shape
    s, t = scores.cpu().numpy(), slots.cpu().numpy()
    os, ot = np.zeros((B, W), np.float32), np.full((B, W), -1, np.int32)
    ol, freed, ptr, status = [], [], [0], 0
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n > S:
            n, status = 0, status | 1
        kept = list(range(n))
        if n > budget:
            mid = list(range(first, n - recent))
            if any(np.isnan(s[b, j]) for j in mid):
                status |= 8
            mid.sort(key=lambda j: (np.isnan(s[b, j]), 0.0 if np.isnan(s[b, j]) else -float(s[b, j]), j))
            kept = sorted(list(range(first)) + mid[:budget - first - recent] + list(range(n - recent, n)))
        os[b, :len(kept)], ot[b, :len(kept)] = s[b, kept], t[b, kept]
        gone = sorted(set(range(n)) - set(kept))
        freed += [int(t[b, j]) for j in gone]
        ptr.append(len(freed))
        ol.append(len(kept))
    return os, ot, ol, freed, ptr, status
