"""Calls of the paged-cache operators that the device refuses: nothing is written."""
import pytest
import torch

import sink_sda_decode_gb300 as sda
from paged_ref import Case
from test_chunk_gpu import KERNELS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,m,K", KERNELS)
def test_bad_lengths_after_a_call_that_cut_units(H, m, K):
    """The merge of cut units is launched for a refused call too.  A workspace that still
    holds the cuts of a larger call (more rows, the same kernel) must not tell it to write:
    out and lse are the beginnings of longer arrays, which stay as they are as well."""
    more = {(4, 1): 2, (64, 1): 1, (64, 5): 4}[H, m]
    big = Case(60, m=[m, m + more], n=[900, 1500], H=H, D=512, K=K)
    c = Case(61, m=[m, m], n=[900, 1500], H=H, D=512, K=K)
    T, rows = 2 * m, big.q.shape[0]
    size = sda.chunk_attention_workspace_size(2, rows, H, 512)
    assert size == sda.chunk_attention_workspace_size(2, T, H, 512)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, H), 7.0, device="cuda")
    for name, value in (("kv_len", [900, 100000]), ("kv_len", [-1, 1500]), ("q_indptr", [0, T + 1, T]),
                        ("q_indptr", [0, m, T + 1]), ("q_indptr", [-1, m, T])):
        big.attend(sda, workspace=ws)
        assert sda.paged_error_flag(ws) == 0
        keep = getattr(c, name)
        setattr(c, name, torch.tensor(value, dtype=torch.int32, device="cuda"))
        c.attend(sda, workspace=ws, out=out[:T], lse=lse[:T])
        assert sda.paged_error_flag(ws) == 2
        setattr(c, name, keep)
        assert bool((out == 7).all()) and bool((lse == 7).all())
    check(c, workspace=ws)
    assert sda.paged_error_flag(ws) == 0


def test_more_tiles_than_are_counted_after_a_call_that_cut_units():
    """64 sequences of 2^31 - 512 positions, each within its bound, are more than 2^31 - 1
    tiles of 48."""
    B, H, D = 64, 64, 512
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, D, device="cuda").to(torch.bfloat16)
    pool = torch.randn(4096, D, device="cuda").to(torch.bfloat16)
    ptr, table = torch.arange(B + 1, **i32), torch.zeros(B, 2, **i32)
    ws = torch.empty(sda.chunk_attention_workspace_size(B, B, H, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((B, H), 7.0, device="cuda")
    for length, error in ((4000, 0), (2 ** 31 - 512, 2)):
        out.fill_(7.0)
        lse.fill_(7.0)
        sda.chunk_attention(q, pool, table, ptr, torch.full((B,), length, **i32), torch.zeros(H, device="cuda"), 0.04,
                            k_per_block=2 ** 30, out=out, lse=lse, workspace=ws)
        assert sda.paged_error_flag(ws) == error
        assert bool((out == 7).all()) == bool(error) and bool((lse == 7).all()) == bool(error)


@pytest.mark.parametrize("what", ["q", "pool", "table", "q_indptr", "kv_len", "sink", "out", "lse", "prev"])
def test_workspace_is_apart(what):
    """A workspace that begins, or ends, inside an array of the call is refused."""
    c = Case(62, m=[2, 3], n=[100, 200], H=16, D=512, K=16)
    lse = torch.zeros(5, 16, device="cuda")
    S = c.table.shape[1] * 16
    sizes = {"attend": sda.chunk_attention_workspace_size(2, 5, 16, 512),
             "mass": sda.attention_mass_workspace_size(2, c.table.shape[1], 16)}

    def call(op, a, ws):
        t = (a.get("q", c.q), a.get("pool", c.pool), a.get("table", c.table), a.get("q_indptr", c.q_indptr),
             a.get("kv_len", c.kv_len))
        if op == "attend":
            sda.chunk_attention(*t, a.get("sink", c.sink), c.scale, k_per_block=16, out=a.get("out"),
                                lse=a.get("lse"), workspace=ws)
        else:
            sda.attention_mass(*t, a.get("lse", lse), c.scale, k_per_block=16, scores=a.get("prev"),
                               out=a.get("out"), workspace=ws)

    for op in ("attend", "mass"):
        if what in {"attend": ("prev",), "mass": ("sink",)}[op]:
            continue
        like = {"out": c.q if op == "attend" else torch.zeros(2, S, device="cuda"), "lse": lse,
                "prev": torch.zeros(2, S, device="cuda")}.get(what)
        like = getattr(c, what) if like is None else like
        n, size = like.numel() * like.element_size(), sizes[op]
        room = (n + 255) // 256 * 256
        buf = torch.zeros(2 * room + size, dtype=torch.uint8, device="cuda")
        for at in (0, (room + size - n) // 256 * 256):  # the array's first byte; the workspace's is room's last 256
            begin = room - 256 if at == 0 else room
            t = buf[at:at + n].view(like.dtype).view(like.shape).copy_(like)
            ws = buf[begin:begin + size]
            overlap = at < begin + size and begin < at + n
            assert overlap
            with pytest.raises(sda._lib.SdaError):
                call(op, {what: t}, ws)
        t = buf[:n].view(like.dtype).view(like.shape).copy_(like)
        call(op, {what: t}, buf[room:room + size])  # one behind the other
        assert sda.paged_error_flag(buf[room:room + size]) == 0
