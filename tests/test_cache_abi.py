"""What the entry points that fill a paged cache, or attend over one in 8 bits, refuse on the
host, before anything is enqueued (CPU only: pointers are fake, and every case is rejected
before any use)."""
import ctypes

import pytest
import torch

import sink_sda_decode_gb300 as sda
from sink_sda_decode_gb300 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from sink_sda_decode_gb300 import build
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def no_gpu(lib):
    """Without a GPU what is accepted gets as far as the device, and no further."""
    if lib.sda_chunk_attention_workspace_size(2, 3, 16, 512, ctypes.byref(ctypes.c_size_t(0))) == OK:
        pytest.skip("would be enqueued")


# every array in a place of its own
ATTEND = dict(q=1 << 40, kv=1 << 41, scale=1 << 42, pages=100, table=1 << 43, max_blocks=4, K=16, base=0,
              indptr=1 << 44, kv_len=1 << 45, sink=1 << 46, softmax=0.1, window=0, first=0, B=2, T=3, H=16, D=512,
              out=1 << 47, lse=1 << 48, ws=1 << 49, bytes=1 << 30)


def attend(lib, **kw):
    a = dict(ATTEND, **kw)
    return lib.sda_chunk_attention_fp8(
        a["q"], a["kv"], a["scale"], a["pages"], a["table"], a["max_blocks"], a["K"], a["base"], a["indptr"],
        a["kv_len"], a["sink"], a["softmax"], a["window"], a["first"], a["B"], a["T"], a["H"], a["D"], a["out"],
        a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(K=0), dict(K=-3), dict(max_blocks=-1), dict(window=-1), dict(first=-1),
    dict(pages=0), dict(pages=1 << 31), dict(base=-1), dict(base=101), dict(T=1 << 27), dict(B=(1 << 24) + 1)]
    + [{name: None} for name in ("q", "kv", "scale", "table", "indptr", "kv_len", "sink", "out", "lse", "ws")]
    + [dict(q=(1 << 40) + 8), dict(kv=(1 << 41) + 8), dict(out=(1 << 47) + 4), dict(lse=(1 << 48) + 2),
       dict(scale=(1 << 42) + 1), dict(indptr=(1 << 44) + 1), dict(table=(1 << 43) + 2)])
def test_chunk_attention_fp8_refuses(lib, bad):
    assert attend(lib, **bad) == INVALID


def test_chunk_attention_fp8_shapes(lib):
    for H, D in ((0, 512), (257, 512), (16, 96), (16, 1024), (16, 0)):
        assert attend(lib, H=H, D=D) == UNSUPPORTED
    assert attend(lib, ws=(1 << 49) + 128) == WORKSPACE
    assert attend(lib, B=0) == OK and attend(lib, T=0) == OK  # nothing to do
    n = ctypes.c_size_t(0)
    size = lib.sda_chunk_attention_fp8_workspace_size
    assert size(1, 1, 16, 512, 0, 1, None) == INVALID
    for bad in ((-1, 1, 16, 512, 0, 1), (1, -1, 16, 512, 0, 1), (1, 1, 16, 512, -1, 1), (1, 1, 16, 512, 4, 0)):
        assert size(*bad, ctypes.byref(n)) == INVALID
    assert size(1, 1, 16, 500, 0, 1, ctypes.byref(n)) == UNSUPPORTED


READS = dict(q=3 * 16 * 1024, kv=100 * 512, scale=7 * 4, table=32, indptr=12, kv_len=8, sink=16 * 4)


@pytest.mark.parametrize("name,size", [*READS.items(), ("out", 3 * 16 * 1024), ("lse", 3 * 16 * 4)])
@pytest.mark.parametrize("result", ["out", "lse"])
def test_results_of_chunk_attention_fp8_are_apart(lib, no_gpu, name, size, result):
    if name == result:
        return
    at, long = ATTEND[name], {"out": 3 * 16 * 1024, "lse": 3 * 16 * 4}[result]
    for where in (at - long + 16, at, at + (size - 1) // 16 * 16):  # 16-byte aligned
        assert attend(lib, **{result: where}) == INVALID
    for where in (at - long, at + -(-size // 16) * 16):
        assert attend(lib, **{result: where}) not in (OK, INVALID)


APPEND = dict(q=1 << 40, kv=1 << 41, q_w=1 << 42, kv_w=1 << 43, cos=1 << 44, sin=1 << 45, max_pos=64,
              table=1 << 46, max_blocks=4, K=16, base=0, indptr=1 << 47, kv_len=1 << 48, B=2, T=3, H=16, D=512,
              rope=64, eps=1e-6, pages=100, q_out=1 << 49, pool=1 << 50, scale=1 << 51, status=1 << 52)
SIZES = dict(q=3 * 16 * 1024, kv=3 * 1024, q_w=1024, kv_w=1024, cos=64 * 32 * 4, sin=64 * 32 * 4, table=32,
             indptr=12, kv_len=8, q_out=3 * 16 * 1024, status=4)


def append(lib, fp8, **kw):
    a = dict(APPEND, **kw)
    args = [a[k] for k in ("q", "kv", "q_w", "kv_w", "cos", "sin", "max_pos", "table", "max_blocks", "K", "base",
                           "indptr", "kv_len", "B", "T", "H", "D", "rope", "eps", "pages", "q_out", "pool")]
    if fp8:
        return lib.sda_append_rows_fp8(*args, a["scale"], a["status"], None)
    return lib.sda_append_rows(*args, a["status"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(H=-1), dict(K=0), dict(K=-1), dict(max_blocks=-1), dict(B=(1 << 24) + 1),
    dict(pages=0), dict(pages=1 << 31), dict(base=-1), dict(base=101), dict(rope=-8), dict(rope=4),
    dict(rope=520), dict(max_pos=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(T=1 << 27, H=16)]
    + [{name: None} for name in ("q", "kv", "cos", "sin", "table", "indptr", "kv_len", "q_out", "pool", "status")]
    + [{name: APPEND[name] + 8} for name in ("q", "kv", "q_w", "kv_w", "cos", "sin", "q_out", "pool")]
    + [{name: APPEND[name] + 2} for name in ("table", "indptr", "kv_len", "status")])
def test_append_refuses(lib, fp8, bad):
    assert append(lib, fp8, **bad) == INVALID


def test_append_refuses_scales(lib):
    assert append(lib, True, scale=None) == INVALID and append(lib, True, scale=(1 << 51) + 2) == INVALID


@pytest.mark.parametrize("fp8", [False, True])
def test_append_widths(lib, fp8):
    for D in (0, 8, 24, 1040, 2048):
        assert append(lib, fp8, D=D, rope=0) == UNSUPPORTED


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", [k for k in SIZES if k not in ("q_out", "status")])
@pytest.mark.parametrize("result", ["q_out", "pool", "status"])
def test_results_of_append_are_apart(lib, no_gpu, fp8, name, result):
    long = {"q_out": 3 * 16 * 1024, "pool": 100 * (512 if fp8 else 1024), "status": 4}[result]
    step = 4 if result == "status" else 16
    at, size = APPEND[name], SIZES[name]
    if (result, name) == ("q_out", "q"):
        assert append(lib, fp8, q_out=at) not in (OK, INVALID)  # in place
        inside = (at - long + step, at + step, at + size - step)
    else:
        inside = (at - long + step if long > step else at, at, at + (size - 1) // step * step)
    for where in inside:
        assert append(lib, fp8, **{result: where}) == INVALID
    for where in (at - long, at + -(-size // step) * step):
        assert append(lib, fp8, **{result: where}) not in (OK, INVALID)


def test_python_refuses(lib):
    t = torch.zeros(2, 4, dtype=torch.int32)
    kv = torch.zeros(3, 64, dtype=torch.bfloat16)
    angles = torch.zeros(8, 16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError, RuntimeError)):  # tensors of the host
        sda.append_rows(kv, angles, angles, t, i, i, k_per_block=16, unified_kv=kv)
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        sda.chunk_attention_fp8(kv.view(3, 1, 64), kv, angles, t, i, i, angles, 1.0, k_per_block=16)
    for bad in ((2 ** 31, 1, 1, 64), (1, 1, 1, 64, 2 ** 31), (1, 1, 1, 64, 1, 0), (1, 1, 1, 64, 1, 2 ** 31)):
        with pytest.raises(ValueError):
            sda.chunk_attention_fp8_workspace_size(*bad)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [1, 16])
@pytest.mark.parametrize("name", ["kv", "q_w", "kv_w", "cos", "sin"])
def test_in_place_is_for_queries_alone(lib, no_gpu, name, H, fp8):
    """q_out = q is taken, but not with another array that is read at the same address: rows of
    it are read by other warps while q's are overwritten."""
    q = APPEND["q"]
    assert append(lib, fp8, H=H, q_out=q) not in (OK, INVALID)
    assert append(lib, fp8, H=H, q_out=q, **{name: q}) == INVALID
    assert append(lib, fp8, H=H, **{name: q}) not in (OK, INVALID)  # read alone: any address
