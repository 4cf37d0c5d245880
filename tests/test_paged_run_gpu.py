"""The paged-cache operators together, as a server would use them: prompts in chunks,
weights accumulated, caches cut down to a budget, then single tokens."""
import numpy as np
import torch
import pytest

import sink_sda_decode_gb300 as sda
from paged_ref import evict

pytestmark = pytest.mark.gpu

H, D, B, BUDGET, FIRST, RECENT, S = 16, 512, 3, 64, 4, 32, 512


def reference(q, rows, sink, scale):
    """One sequence in 64 bits: q [m, H, D] over its rows [n, D], the last m its own."""
    m, n = q.shape[0], rows.shape[0]
    x = torch.einsum("thd,jd->thj", q, rows) * scale
    see = torch.arange(n)[None] <= torch.arange(n - m, n)[:, None]
    x = torch.where(see[:, None], x, torch.full_like(x, -float("inf")))
    z = torch.logsumexp(torch.cat([x, sink.view(1, H, 1).expand(m, H, 1)], 2), dim=2)
    w = torch.exp(x - z[..., None])
    return torch.einsum("thj,jd->thd", w, rows), w.sum(dim=(0, 1))


def test_prompts_then_eviction_then_steps():
    g = torch.Generator().manual_seed(1)
    scale = D ** -0.5
    sink = torch.randn(H, generator=g)
    pool = torch.zeros(B * S, D, dtype=torch.bfloat16, device="cuda")
    free = torch.randperm(B * S, generator=g).tolist()
    table = torch.full((B, S), -1, dtype=torch.int32, device="cuda")
    scores = torch.zeros(B, S, device="cuda")
    rows = [torch.zeros(0, D, dtype=torch.float64) for _ in range(B)]   # what each cache holds, in 64 bits
    ref_scores = [torch.zeros(0, dtype=torch.float64) for _ in range(B)]
    chunks = [[90, 150, 40], [60, 1, 33], [1, 1, 1], [1, 1, 1], [5, 1, 2], [1, 1, 1]]
    evictions = 0
    for ms in chunks:
        q = torch.randn(sum(ms), H, D, generator=g).to(torch.bfloat16)
        new = [torch.randn(m, D, generator=g).to(torch.bfloat16) for m in ms]
        for b, m in enumerate(ms):  # the chunk's own rows into free slots
            slots = [free.pop() for _ in range(m)]
            n = rows[b].shape[0]
            pool[slots] = new[b].cuda()
            table[b, n:n + m] = torch.tensor(slots, dtype=torch.int32)
            rows[b] = torch.cat([rows[b], new[b].double()])
            ref_scores[b] = torch.cat([ref_scores[b], torch.zeros(m, dtype=torch.float64)])
        lens = torch.tensor([r.shape[0] for r in rows], dtype=torch.int32, device="cuda")
        ptr = torch.tensor(np.cumsum([0] + ms), dtype=torch.int32, device="cuda")
        qd = q.cuda()
        out, lse = sda.chunk_attention(qd, pool, table, ptr, lens, sink.cuda(), scale, k_per_block=1)
        scores = sda.attention_mass(qd, pool, table, ptr, lens, lse, scale, k_per_block=1, scores=scores,
                                    out=scores)
        for b, m in enumerate(ms):
            s = slice(int(ptr[b]), int(ptr[b + 1]))
            o, w = reference(q[s].double(), rows[b], sink.double(), scale)
            # |out| < 6: half a bf16 step of it and of the weights, 2^-8 each, twice over
            assert float((out[s].double().cpu() - o).abs().max()) <= 2 * 2.0 ** -8 * 6
            ref_scores[b] = ref_scores[b] + w
            n = rows[b].shape[0]
            assert torch.allclose(scores[b, :n].double().cpu(), ref_scores[b], rtol=1e-4, atol=1e-6)
            assert bool((scores[b, n:] == 0).all())
        # the kernel's own numbers decide, exactly
        want = evict(scores, table, lens.tolist(), BUDGET, FIRST, RECENT, S)
        r = sda.evict_slots(scores, table, lens, BUDGET, first=FIRST, recent=RECENT)
        W = min(S, BUDGET)
        assert np.array_equal(r.slot_table.cpu().numpy(), want[1][:, :W])
        assert r.kv_len.tolist() == want[2] and int(r.status.item()) == 0
        n_freed = int(r.freed_indptr[-1])
        evictions += n_freed
        old = table.cpu().numpy()
        for b in range(B):  # the same rows kept on this side
            kept = [int(np.flatnonzero(old[b, :rows[b].shape[0]] == s)[0]) for s in want[1][b, :want[2][b]]]
            rows[b] = rows[b][kept]
            ref_scores[b] = ref_scores[b][kept]
        free += r.freed_slots[:n_freed].tolist()
        table[:, :W], table[:, W:] = r.slot_table, -1
        scores = torch.cat([r.scores, torch.zeros(B, S - W, device="cuda")], dim=1)
    assert evictions > 100
    # what is left is read by decode() too: its lists are the kept slots
    n = [x.shape[0] for x in rows]
    idx = torch.cat([table[b, :n[b]] for b in range(B)])
    ptr = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, D, generator=g).to(torch.bfloat16)
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    a, _ = sda.chunk_attention(q.cuda(), pool, table, one, lens, sink.cuda(), scale, k_per_block=1)
    d = sda.decode(q.cuda(), pool, idx, ptr, sink.cuda(), scale)
    assert float((a.double() - d.double()).abs().max()) <= 4 * 2.0 ** -8 * 6


@pytest.mark.parametrize("B,T", [(0, 0), (2, 0)])
def test_error_word_of_calls_without_work(B, T):
    """0, whatever the workspace held before."""
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(T, 16, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    ptr, n = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    ws = torch.full((max(sda.chunk_attention_workspace_size(B, T, 16, 64),
                         sda.attention_mass_workspace_size(B, 0, 16)),), 0x7f, dtype=torch.uint8, device="cuda")
    _, lse = sda.chunk_attention(q, pool, torch.zeros(B, 1, **i32), ptr, n, torch.zeros(16, device="cuda"), 0.1,
                                 k_per_block=16, workspace=ws)
    assert sda.paged_error_flag(ws) == 0
    ws.fill_(0x7f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sda.attention_mass(q, pool, torch.zeros(B, 0, **i32), ptr, n, lse, 0.1, k_per_block=16, workspace=ws, stream=side)
    assert sda.paged_error_flag(ws, side) == 0


def test_error_word_needs_a_workspace():
    with pytest.raises(ValueError):
        sda.paged_error_flag(torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        sda.paged_error_flag(torch.zeros(1 << 20, device="cuda"))


@pytest.mark.parametrize("op", ["attend", "mass", "evict"])
def test_results_on_another_stream_are_not_given_away(op):
    """Results that are dropped while their call still waits on its stream."""
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(64, 16, 512, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(4096, 512, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(4096, **i32).view(1, 4096)
    ptr, n = torch.tensor([0, 64], **i32), torch.tensor([4096], **i32)
    lse, scores = torch.zeros(64, 16, device="cuda"), torch.zeros(1, 4096, device="cuda")
    sink = torch.zeros(16, device="cuda")
    side = torch.cuda.Stream()

    def call():
        if op == "attend":
            return sda.chunk_attention(q, pool, table, ptr, n, sink, 0.1, k_per_block=1, stream=side)
        if op == "mass":
            return (sda.attention_mass(q, pool, table, ptr, n, lse, 0.1, k_per_block=1, stream=side),)
        return tuple(sda.evict_slots(scores, table, n, 1000, stream=side))

    call()  # (what is made once)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    gate = torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # 0.1 s: the call waits behind it
    r = call()
    gate.record(side)
    like = [(t.shape, t.dtype, t.data_ptr()) for t in r]
    del r
    again = [torch.empty(s, dtype=d, device="cuda") for s, d, _ in like]
    assert not gate.query()  # still waiting
    assert not {t.data_ptr() for t in again} & {p for _, _, p in like}
    torch.cuda.synchronize()
