"""Memory that a call on another stream makes for itself: a block that was freed on the
current stream, where queued work still uses it, is not written by the call."""
import pytest
import torch

import parity
import sink_sda_decode_gb300 as sda
from sink_sda_decode_gb300 import inputs

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def paged():
    q = torch.randn(64, 16, 512, device="cuda").to(torch.bfloat16)
    pool = torch.randn(4096, 512, device="cuda").to(torch.bfloat16)
    table = torch.arange(4096, **I32).view(1, 4096)
    ptr, n = torch.tensor([0, 64], **I32), torch.tensor([4096], **I32)
    lse, scores = torch.zeros(64, 16, device="cuda"), torch.rand(1, 4096, device="cuda")
    sink = torch.zeros(16, device="cuda")
    attend = lambda s: sda.chunk_attention(q, pool, table, ptr, n, sink, 0.04, k_per_block=1, stream=s)
    return {"attend": attend,
            "mass": lambda s: (sda.attention_mass(q, pool, table, ptr, n, lse, 0.04, k_per_block=1, stream=s),),
            "evict": lambda s: tuple(sda.evict_slots(scores, table, n, 1000, stream=s))}


def check_untouched(call):
    """Copies of what lay in the call's own blocks before, made by work that is queued on
    the current stream when the blocks are freed and the call runs on another."""
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    call(side)  # (what is made once)
    torch.cuda.synchronize()
    before = [torch.full_like(t, 3) for t in want]
    ws = torch.full((64 << 20,), 3, dtype=torch.uint8, device="cuda")  # workspaces are cut from it, if from any
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # 0.2 s: the copies wait behind it
    copies = [t.clone() for t in before + [ws]]
    del before, ws
    got = call(side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the copies are still to be made
    torch.cuda.synchronize()
    for t in copies:
        assert bool((t == 3).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def check_not_given_away(call):
    """A result that is dropped while work on the current stream still reads it."""
    want = call(None)[0].clone()
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    got = call(side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(400_000_000)
    copy = got.clone()
    shape, dtype = got.shape, got.dtype
    del got
    with torch.cuda.stream(side):
        torch.full(shape, 3, dtype=dtype, device="cuda")
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("op", ["attend", "mass", "evict"])
def test_paged_operators(op):
    check_untouched(paged()[op])
    check_not_given_away(paged()[op])


def test_two_calls_without_a_workspace_on_two_streams():
    """The first call's workspace is dropped, its kernels still to run, when the second
    call makes its own."""
    call = paged()["attend"]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(20_000_000)
        a = call(None)
        b = call(side)
        torch.cuda.synchronize()
        for x in (a, b):
            assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])


def path(op):
    """The calls of the decode path, with the part of each result that is defined whole."""
    w = inputs.config(1, device="cuda")
    if op == "decode":
        idx, ptr = parity.to_dev(w)
        return lambda s: (sda.decode(w.q, w.unified_kv, idx, ptr, w.attn_sink, w.softmax_scale, stream=s),)
    if op == "fp8":
        idx, ptr = parity.to_dev(w)
        pool = inputs.fp8_pool(w)
        return lambda s: (sda.decode_fp8(w.q, pool.codes, pool.scale, idx, ptr, w.attn_sink, w.softmax_scale,
                                         stream=s),)
    if op in ("build", "build_decode"):
        bi = w.builder_inputs("cuda")
        kw = dict(win=w.win, k_per_block=w.k_per_block, swa_pages=w.swa_pages)
        if op == "build":
            return lambda s: sda.build_indices(**bi, **kw, total_pages=w.total_pages, stream=s)[1:]
        names = ("state_slot", "swa_len", "swa_head", "comp_indptr", "comp_block", "comp_slot")
        return lambda s: sda.build_decode(w.q, w.unified_kv, w.attn_sink, w.softmax_scale, *(bi[x] for x in names),
                                          **kw, stream=s)[::2]
    if op == "topk":
        ti = inputs.topk_inputs(w)
        return lambda s: sda.topk_slots(ti.scores, ti.lengths, ti.block_table, k=ti.k, k_per_block=w.k_per_block,
                                        stream=s)[::3]
    si = inputs.store_inputs(w)
    return lambda s: sda.qk_norm_rope_swa_store(w.q, si.kv_new, si.q_norm_w, si.kv_norm_w, si.cos_cache, si.sin_cache,
                                                si.positions, si.state_slot, eps=si.eps, win=w.win,
                                                swa_pages=w.swa_pages, unified_kv=w.unified_kv, stream=s)


@pytest.mark.parametrize("op", ["decode", "fp8", "build", "build_decode", "topk", "store"])
def test_decode_path(op):
    check_untouched(path(op))
    check_not_given_away(path(op))


def test_error_word_of_decode_on_another_stream():
    """It is that of the call, also while the call still waits on its stream."""
    w = inputs.random_small(seed=90, N=2, H=16, D=512, P=100, lengths=[3, 4], device="cuda")
    idx, ptr = parity.to_dev(w)
    ws = torch.empty(sda.workspace_size(w.N, w.H, w.D, idx.numel()), dtype=torch.uint8, device="cuda")
    bad = torch.tensor([0, 5, 4], **I32)  # no prefix sums
    side = torch.cuda.Stream()
    for p, word in ((bad, 2), (ptr, 0)):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        sda.decode(w.q, w.unified_kv, idx, p, w.attn_sink, w.softmax_scale, workspace=ws, stream=side)
        assert sda.decode_error_flag(ws, side) == word


@pytest.mark.parametrize("op", ["attend", "mass", "evict", "decode"])
def test_captured_on_a_forked_stream(op):
    """A call without memory of its own on a stream that a capture has forked."""
    call = path(op) if op == "decode" else paged()[op]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
