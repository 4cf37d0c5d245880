"""The paged-cache operators: inputs, plain forms and sizes of what is measured.

Three operators work on a cache whose rows lie in one pool (a row is key and
value of a position) and are found through a table per sequence:

* attend  -- a chunk of new tokens of every sequence over its cached positions,
             causal, optionally with a sliding window and a few first positions
             that stay visible, with a sink logit per head;
* mass    -- the attention weight that every cached position received from the
             chunk's tokens, added to what it had;
* evict   -- which positions of each sequence to keep by that weight, with the
             slots that become free.

With m_b new tokens and n_b cached positions (the new tokens' own rows are the
last m_b of them), token i of sequence b stands at position p = n_b - m_b + i and
sees position j if j <= p and (window = 0, or p - j < window, or j < first).
"""
import math
import random

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def _case(name, op, B, H=0, D=0, K=1, m=(1, 1), n=(1, 1), window=0, first=0, budget=0, recent=0):
    return {"name": name, "op": op, "B": B, "H": H, "D": D, "K": K, "m_lo": m[0], "m_hi": m[1],
            "n_lo": n[0], "n_hi": n[1], "window": window, "first": first, "budget": budget,
            "recent": recent}


def listed():
    return [
        # one new token per sequence over a few hundred cached rows: a small decode batch
        _case("attend_step", "attend", 64, 16, 512, 64, (1, 1), (513, 767)),
        # one new token per sequence over long caches: a few long conversations
        _case("attend_long_step", "attend", 8, 64, 512, 64, (1, 1), (16384, 65536)),
        # a few drafted tokens to verify, cache held as single slots after evictions
        _case("attend_verify", "attend", 32, 128, 512, 1, (2, 5), (1000, 4096)),
        # prompts of mixed lengths, some with a cached prefix
        _case("attend_ragged", "attend", 12, 64, 512, 64, (1, 300), (300, 6000)),
        # a chunk of a long prompt behind three chunks that are cached
        _case("attend_prompt", "attend", 1, 64, 512, 64, (2048, 2048), (8192, 8192)),
        # prompts with a sliding window of 128 and four first positions that stay visible
        _case("attend_window", "attend", 4, 64, 512, 64, (700, 1000), (1000, 5000), 128, 4),
        # a small head layout, a handful of tokens: a unit-test sized model
        _case("attend_tiny", "attend", 4, 8, 64, 16, (1, 17), (17, 130)),
        # weights of one step of a small decode batch
        _case("mass_step", "mass", 64, 16, 512, 1, (1, 1), (513, 767)),
        # weights of one step over long caches
        _case("mass_long_step", "mass", 8, 64, 512, 64, (1, 1), (16384, 65536)),
        # weights of a prompt chunk, to rank its positions before the first eviction
        _case("mass_chunk", "mass", 2, 64, 512, 64, (500, 600), (6000, 8192)),
        # a decode batch that has grown past its budget of 512 rows by a window
        _case("evict_step", "evict", 64, n=(500, 768), first=4, budget=512, recent=128),
        # long prompts cut down to a budget
        _case("evict_prompt", "evict", 16, n=(8000, 131072), first=4, budget=4096, recent=128),
    ]


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["attend", "attend", "attend", "mass", "mass", "evict"])
        if op == "evict":
            B = _log_int(rng, 1, 64)
            hi = _log_int(rng, 130, 131072)
            lo = _log_int(rng, max(1, hi // 16), hi)
            budget = _log_int(rng, max(1, lo // 8), hi)
            first = rng.choice([0, 1, 4])
            recent = rng.randint(0, min(128, budget))
            if first + recent > budget or B * hi > 16 * 131072:
                continue
            return _unnamed(_case("", op, B, n=(lo, hi), first=first, budget=budget, recent=recent))
        B = _log_int(rng, 1, 64)
        H = rng.choice([1, 5, 8, 16, 24, 32, 64, 64, 128])
        D = rng.choice([64, 128, 256, 512, 512, 512])
        K = rng.choice([1, 16, 64, 64, 100])
        m_hi = rng.choice([1, 1, _log_int(rng, 2, 2048)])
        m_lo = rng.choice([m_hi, _log_int(rng, 1, m_hi)])
        n_hi = max(m_hi, _log_int(rng, 64, 65536))
        n_lo = rng.choice([n_hi, max(m_hi, _log_int(rng, max(1, n_hi // 8), n_hi))])
        window, first = rng.choice([(0, 0), (0, 0), (rng.randint(1, 512), rng.choice([0, 1, 4, 70]))])
        rows = B * m_hi * H
        if rows * n_hi > 3 << 28 or rows > 1 << 18 or B * n_hi > 1 << 19:
            continue
        return _unnamed(_case("", op, B, H, D, K, (m_lo, m_hi), (n_lo, n_hi), window, first))


def _lengths(case):
    """(new tokens, cached positions) of every sequence: a function of the case alone."""
    r = random.Random(case["B"] * 7919 + case["n_hi"] * 31 + case["m_hi"])
    m = [r.randint(case["m_lo"], case["m_hi"]) for _ in range(case["B"])]
    n = [max(r.randint(case["n_lo"], case["n_hi"]), x) for x in m]
    n[r.randrange(case["B"])] = max(case["n_hi"], max(m))
    return m, n


def _visible(m, n, window, first):
    """Pairs (token, position) that attend, and the positions that any token sees."""
    pairs = seen = 0
    for a, b in zip(m, n):
        p = np.arange(b - a, b, dtype=np.int64)
        if window == 0:
            pairs += int((p + 1).sum())
            seen += b
        else:
            lo = np.maximum(p - window + 1, 0)
            pairs += int((p + 1 - lo + np.minimum(first, lo)).sum())
            seen += b - int(lo[0]) + min(first, int(lo[0]))
    return pairs, seen


def work(case):
    m, n = _lengths(case)
    B, H, D = case["B"], case["H"], case["D"]
    if case["op"] == "evict":
        # a sequence within its budget is copied; one above it has its scores and
        # slots read, the kept ones written and the others' slots written
        kept = sum(min(x, case["budget"]) for x in n)
        return {"bytes": 8 * sum(n) + 8 * kept + 4 * (sum(n) - kept) + 12 * B, "flops": sum(n)}
    pairs, seen = _visible(m, n, case["window"], case["first"])
    T = sum(m)
    table = 4 * sum(-(-x // case["K"]) for x in n)
    if case["op"] == "attend":
        return {"bytes": 2 * D * seen + 4 * D * T * H + 4 * T * H + table + 4 * H,
                "flops": 4 * H * D * pairs}
    return {"bytes": 2 * D * seen + 2 * D * T * H + 4 * T * H + table + 8 * sum(n),
            "flops": 2 * H * D * pairs}


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed * 1000003 + 17)
    m, n = _lengths(case)
    B, H, D, K = case["B"], case["H"], case["D"], case["K"]
    st = {"case": case, "n": torch.tensor(n, dtype=torch.int32, device=dev), "n_max": max(n),
          "m_max": max(m), "m": torch.tensor(m, dtype=torch.int64, device=dev)}
    if case["op"] == "evict":
        S = max(n)
        # accumulated weights fall off over the cache and differ widely between positions
        st["scores"] = torch.exp(1.5 * torch.randn(B, S, generator=g, device=dev)) / 64
        st["slots"] = torch.randperm(B * S, generator=g, device=dev).to(torch.int32).view(B, S)
        return st
    blocks = [-(-x // K) for x in n]
    mb = max(blocks)
    total = sum(blocks) + 3
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, mb, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    T = sum(m)
    st["table"] = table
    st["pool"] = torch.randn(total * K, D, generator=g, device=dev).to(torch.bfloat16)
    st["q"] = torch.randn(T, H, D, generator=g, device=dev).to(torch.bfloat16)
    st["sink"] = torch.randn(H, generator=g, device=dev)
    st["q_indptr"] = torch.tensor(np.cumsum([0] + m), dtype=torch.int32, device=dev)
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "mass":
        st["lse"] = _plain_attend(st)["lse"]
        st["scores"] = torch.rand(B, mb * K, generator=g, device=dev) * 4
    return st


# --------------------------------------------------------------- plain forms
def _plain_scores(st):
    """Scaled scores [B, m_max, H, n_max] of the padded chunks (masked: -inf), the
    cached rows in 32 bits [B, n_max, D], and the token of every padded row."""
    case = st["case"]
    K, B = case["K"], case["B"]
    H, D = st["q"].shape[1:]
    j = torch.arange(st["n_max"], device="cuda")
    slot = st["table"][:, j // K].long() * K + j % K
    n = st["n"].long()
    slot = torch.where(j[None] < n[:, None], slot, 0)
    kv = st["pool"][slot].float()
    i = torch.arange(st["m_max"], device="cuda")
    tok = torch.minimum(st["q_indptr"][:-1].long()[:, None] + i[None], st["q_indptr"][-1].long() - 1)
    qp = st["q"][tok].float().reshape(B, -1, D)
    x = torch.matmul(qp, kv.transpose(1, 2)).view(B, st["m_max"], H, st["n_max"]) * st["scale"]
    pos = (n - st["m"])[:, None] + i[None]
    see = j[None, None] <= pos[:, :, None]
    if case["window"]:
        see &= (pos[:, :, None] - j[None, None] < case["window"]) | (j[None, None] < case["first"])
    real = i[None] < st["m"][:, None]
    see &= real[:, :, None]
    x.masked_fill_(~see[:, :, None, :], -math.inf)
    return x, kv, real


def _plain_attend(st):
    x, kv, real = _plain_scores(st)
    B, mm, H, _ = x.shape
    sink = st["sink"].view(1, 1, H, 1)
    top = torch.maximum(x.amax(dim=3, keepdim=True), sink)
    p = torch.exp(x.sub_(top))
    den = p.sum(dim=3, keepdim=True) + torch.exp(sink - top)
    o = torch.matmul(p.view(B, mm * H, -1), kv).view(B, mm, H, -1) / den
    lse = (top + torch.log(den)).squeeze(3)
    return {"out": o[real].to(torch.bfloat16), "lse": lse[real].contiguous()}


def _plain_mass(st):
    x, _, real = _plain_scores(st)
    B, mm, H, n_max = x.shape
    lse = torch.zeros(B, mm, H, device="cuda")
    lse[real] = st["lse"]
    p = torch.exp(x.sub_(lse[..., None]))
    add = p.view(B, mm * H, n_max).sum(dim=1)
    live = torch.arange(st["scores"].shape[1], device="cuda")[None] < st["n"][:, None]
    out = torch.where(live, st["scores"], 0.0)
    out[:, :n_max] += add
    return out


def _plain_evict(st):
    case = st["case"]
    s, slots, n = st["scores"], st["slots"], st["n"].long()
    B, S = s.shape
    j = torch.arange(S, device="cuda")[None].expand(B, S)
    live = j < n[:, None]
    keep_n = torch.clamp(n, max=case["budget"])
    held = (j < case["first"]) | (j >= n[:, None] - case["recent"])
    # larger score first, equal scores by position: NaN counts below every number
    rank = torch.where(torch.isnan(s), -math.inf, s).double()
    rank = torch.where(held, math.inf, rank)
    rank = torch.where(live, rank, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(1, order, j.contiguous())
    kept = live & (place < keep_n[:, None])
    gone = live & ~kept
    W = min(S, case["budget"])
    to = torch.where(kept, kept.long().cumsum(1) - 1, W)
    new_s = torch.zeros(B, W + 1, device="cuda").scatter_(1, to, s)
    new_t = torch.full((B, W + 1), -1, dtype=torch.int32, device="cuda").scatter_(1, to, slots)
    fill = torch.arange(W, device="cuda")[None] < keep_n[:, None]
    new_s = torch.where(fill, new_s[:, :W], 0.0)
    new_t = torch.where(fill, new_t[:, :W], -1)
    indptr = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    indptr[1:] = torch.cumsum(n - keep_n, 0)
    freed = torch.full((B * max(S - case["budget"], 0) + 1,), -1, dtype=torch.int32, device="cuda")
    at = torch.where(gone, indptr[:-1].long()[:, None] + gone.long().cumsum(1) - 1, freed.numel() - 1)
    freed.scatter_(0, at.flatten(), slots.flatten())
    freed = freed[:-1]
    freed = torch.where(torch.arange(freed.numel(), device="cuda") < indptr[-1], freed, -1)
    return {"scores": new_s, "slots": new_t, "len": keep_n.to(torch.int32), "freed": freed,
            "freed_indptr": indptr}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import sink_sda_decode_gb300 as sda
        if op == "attend":
            out, lse = sda.chunk_attention(
                state["q"], state["pool"], state["table"], state["q_indptr"], state["n"],
                state["sink"], state["scale"], k_per_block=case["K"], window=case["window"],
                first=case["first"])
            return {"out": out, "lse": lse}
        if op == "mass":
            return {"scores": sda.attention_mass(
                state["q"], state["pool"], state["table"], state["q_indptr"], state["n"],
                state["lse"], state["scale"], k_per_block=case["K"], window=case["window"],
                first=case["first"], scores=state["scores"])}
        r = sda.evict_slots(state["scores"], state["slots"], state["n"], case["budget"],
                            first=case["first"], recent=case["recent"])
        return {"scores": r.scores, "slots": r.slot_table, "len": r.kv_len, "freed": r.freed_slots,
                "freed_indptr": r.freed_indptr}
    if op == "attend":
        return _plain_attend(state)
    if op == "mass":
        return {"scores": _plain_mass(state)}
    return _plain_evict(state)


# --------------------------------------------------------------- definitions
def exact(case, seed):
    """The operators' definitions, sequence by sequence and block of tokens by block
    of tokens, in 64 bits."""
    st = prepare(case, seed)
    m, n = _lengths(case)
    if case["op"] == "evict":
        return _exact_evict(st, n)
    K = case["K"]
    pool, q, table = st["pool"].double(), st["q"].double(), st["table"].cpu().numpy()
    T, H, D = q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mass = st["scores"].double() if case["op"] == "mass" else None
    sink = st["sink"].double()
    t0 = 0
    for b, (mb, nb) in enumerate(zip(m, n)):
        at = np.arange(nb)
        rows = pool[torch.from_numpy(table[b][at // K].astype(np.int64) * K + at % K).cuda()]
        if mass is not None:
            mass[b, nb:] = 0
        step = max(1, (1 << 27) // (H * nb))
        for i0 in range(0, mb, step):
            i1 = min(mb, i0 + step)
            p = np.arange(nb - mb + i0, nb - mb + i1)
            see = at[None] <= p[:, None]
            if case["window"]:
                see = see & ((at[None] > p[:, None] - case["window"]) | (at[None] < case["first"]))
            see = torch.from_numpy(see).cuda()
            x = torch.einsum("thd,jd->htj", q[t0 + i0:t0 + i1], rows) * st["scale"]
            x = torch.where(see[None], x, -math.inf)
            if mass is not None:
                w = torch.exp(x - st["lse"][t0 + i0:t0 + i1].double().t()[:, :, None])
                mass[b, :nb] += w.sum(dim=(0, 1))
                continue
            z = torch.logsumexp(torch.cat([x, sink.view(H, 1, 1).expand(H, i1 - i0, 1)], 2), dim=2)
            w = torch.exp(x - z[:, :, None])
            out[t0 + i0:t0 + i1] = torch.einsum("htj,jd->thd", w, rows)
            lse[t0 + i0:t0 + i1] = z.t()
        t0 += mb
    return {"scores": mass} if mass is not None else {"out": out, "lse": lse}


def _exact_evict(st, n):
    """Python's own sort of (held first, score falling, position rising)."""
    case = st["case"]
    s, t = st["scores"].cpu().numpy(), st["slots"].cpu().numpy()
    B, S = s.shape
    W = min(S, case["budget"])
    scores = np.zeros((B, W))
    for b in range(B):
        j = np.arange(n[b])
        held = (j < case["first"]) | (j >= n[b] - case["recent"])
        order = np.lexsort((j, -s[b, :n[b]].astype(np.float64), ~held))
        kept = np.sort(order[:case["budget"]])
        scores[b, :len(kept)] = s[b, kept]
    return {"scores": torch.from_numpy(scores).cuda(), "slots": None, "len": None, "freed": None,
            "freed_indptr": None}
