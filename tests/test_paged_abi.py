"""What the paged-cache entry points refuse on the host, before anything is enqueued
(CPU only: pointers are fake, and every case is rejected before any use)."""
import ctypes

import pytest

import sink_sda_decode_gb300 as sda
from sink_sda_decode_gb300 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from sink_sda_decode_gb300 import build
    build.build()
    return _lib.load()


ATTEND = dict(q=1 << 20, kv=1 << 24, pages=100, table=16, max_blocks=4, K=16, base=0, indptr=16, kv_len=16,
              sink=16, scale=0.1, window=0, first=0, B=2, T=3, H=16, D=512, out=1 << 22, lse=16, ws=256,
              bytes=1 << 30)


def attend(lib, **kw):
    a = dict(ATTEND, **kw)
    return lib.sda_chunk_attention(a["q"], a["kv"], a["pages"], a["table"], a["max_blocks"], a["K"],
                                   a["base"], a["indptr"], a["kv_len"], a["sink"], a["scale"],
                                   a["window"], a["first"], a["B"], a["T"], a["H"], a["D"], a["out"],
                                   a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(K=0), dict(K=-3), dict(max_blocks=-1), dict(window=-1), dict(first=-1),
    dict(pages=0), dict(pages=1 << 31), dict(base=-1), dict(base=101), dict(T=1 << 27),
    dict(B=(1 << 24) + 1), dict(q=None), dict(kv=None), dict(table=None), dict(indptr=None),
    dict(kv_len=None), dict(sink=None), dict(out=None), dict(lse=None), dict(ws=None), dict(q=(1 << 20) + 8),
    dict(kv=(1 << 24) + 2), dict(out=(1 << 22) + 4), dict(lse=18), dict(indptr=17),
    dict(out=1 << 20), dict(out=(1 << 20) + 1024), dict(out=1 << 24)])
def test_chunk_attention_refuses(lib, bad):
    assert attend(lib, **bad) == INVALID


def test_chunk_attention_shapes(lib):
    for H, D in ((0, 512), (257, 512), (16, 96), (16, 1024), (16, 0)):
        assert attend(lib, H=H, D=D) == UNSUPPORTED
    assert attend(lib, ws=128) == WORKSPACE
    assert attend(lib, B=0) == OK and attend(lib, T=0) == OK  # nothing to do
    n = ctypes.c_size_t(0)
    assert lib.sda_chunk_attention_workspace_size(1, 1, 16, 512, None) == INVALID
    assert lib.sda_chunk_attention_workspace_size(-1, 1, 16, 512, ctypes.byref(n)) == INVALID
    assert lib.sda_chunk_attention_workspace_size(1, 1, 16, 500, ctypes.byref(n)) == UNSUPPORTED


MASS = dict(q=1 << 20, kv=1 << 24, pages=100, table=16, max_blocks=4, K=16, base=0, indptr=16, kv_len=16,
            lse=16, scale=0.1, window=0, first=0, prev=None, decay=1.0, B=2, T=3, H=16, D=512, out=1 << 22,
            ws=256, bytes=1 << 30)


def mass(lib, **kw):
    a = dict(MASS, **kw)
    return lib.sda_attention_mass(a["q"], a["kv"], a["pages"], a["table"], a["max_blocks"], a["K"],
                                  a["base"], a["indptr"], a["kv_len"], a["lse"], a["scale"], a["window"],
                                  a["first"], a["prev"], a["decay"], a["B"], a["T"], a["H"], a["D"],
                                  a["out"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(K=0), dict(window=-1), dict(first=-1), dict(pages=0), dict(base=101),
    dict(q=None), dict(lse=None), dict(kv=None), dict(table=None), dict(out=None), dict(ws=None),
    dict(q=(1 << 20) + 8), dict(out=(1 << 22) + 2), dict(prev=(1 << 22) + 16), dict(prev=17),
    dict(max_blocks=1 << 20, K=1 << 20), dict(max_blocks=1 << 24, K=64, B=1 << 10)])
def test_attention_mass_refuses(lib, bad):
    assert mass(lib, **bad) == INVALID


def test_attention_mass_shapes(lib):
    assert mass(lib, H=300) == UNSUPPORTED and mass(lib, D=100) == UNSUPPORTED
    assert mass(lib, ws=64) == WORKSPACE
    assert mass(lib, B=0) == OK and mass(lib, max_blocks=0) == OK
    assert lib.sda_attention_mass_workspace_size(1, 1, 16, None) == INVALID
    assert lib.sda_paged_error_flag(None, 16, None) == INVALID
    assert lib.sda_paged_error_flag(256, None, None) == INVALID


EVICT = dict(scores=1 << 20, table=1 << 21, stride=700, kv_len=16, B=4, budget=512, first=4, recent=128,
             out_scores=1 << 22, out_table=1 << 23, out_stride=512, out_len=64, freed=1 << 24,
             capacity=4 * 188, indptr=256, status=512)


def evict(lib, **kw):
    a = dict(EVICT, **kw)
    return lib.sda_evict_slots(a["scores"], a["table"], a["stride"], a["kv_len"], a["B"], a["budget"],
                               a["first"], a["recent"], a["out_scores"], a["out_table"], a["out_stride"],
                               a["out_len"], a["freed"], a["capacity"], a["indptr"], a["status"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(stride=-1), dict(stride=1 << 31), dict(budget=-1), dict(first=-1), dict(recent=-1),
    dict(first=400, recent=113), dict(out_stride=511), dict(capacity=4 * 188 - 1), dict(capacity=-1),
    dict(scores=None), dict(table=None), dict(kv_len=None), dict(out_scores=None), dict(out_table=None),
    dict(out_len=None), dict(freed=None), dict(indptr=None), dict(status=None), dict(scores=(1 << 20) + 1),
    dict(out_scores=(1 << 20)), dict(out_scores=(1 << 20) + 400), dict(out_table=(1 << 21) + 4),
    dict(out_len=20)])
def test_evict_slots_refuses(lib, bad):
    assert evict(lib, **bad) == INVALID


@pytest.mark.parametrize("lse", [1 << 20, (1 << 20) + 3 * 16 * 1024 - 4, 1 << 24, 1 << 22, (1 << 22) - 188])
def test_lse_of_chunk_attention_is_apart(lib, lse):
    """From q, the pool and out (3 x 16 rows)."""
    assert attend(lib, lse=lse) == INVALID
    assert attend(lib, lse=(1 << 22) - 192, ws=128) == WORKSPACE  # ends where out begins


@pytest.mark.parametrize("bad", [dict(out=1 << 20), dict(out=(1 << 20) - 508), dict(out=(1 << 24) + 16),
                                 dict(lse=(1 << 22) + 64), dict(table=(1 << 22) - 28)])
def test_out_of_attention_mass_is_apart(lib, bad):
    assert mass(lib, **bad) == INVALID
    assert mass(lib, prev=1 << 22, ws=64) == WORKSPACE  # in place


@pytest.mark.parametrize("bad", [
    dict(freed=1 << 20), dict(freed=(1 << 21) + 64), dict(freed=(1 << 22) + 4), dict(out_table=1 << 20),
    dict(out_scores=1 << 21), dict(out_table=1 << 22), dict(out_len=(1 << 20) + 8), dict(indptr=12),
    dict(status=20), dict(status=64), dict(status=256 + 16), dict(indptr=60), dict(out_stride=700, out_table=1 << 20),
    dict(out_stride=700, out_scores=1 << 21)])
def test_results_of_evict_slots_are_apart(lib, bad):
    assert evict(lib, **bad) == INVALID


@pytest.mark.parametrize("K,refused", [(1, True), (511, True), (512, False)])
def test_attention_mass_rows_end_within_32_bits(lib, K, refused):
    """Rows of 2^31 - K positions."""
    n = ctypes.c_size_t(0)
    a = (1, 1, 2 ** 31 - K, ctypes.byref(n))
    got = lib.sda_attention_mass_workspace_size(*a)
    assert (got == INVALID) if refused else (got != INVALID)  # (without a GPU no size is known)


def test_python_refuses_sizes_that_do_not_fit():
    with pytest.raises(ValueError):
        sda.chunk_attention_workspace_size(2 ** 31, 1, 1, 64)
    with pytest.raises(ValueError):
        sda.attention_mass_workspace_size(1, 1, 0)


# every array in a place of its own, 1 MB apart at least: (pointer, bytes)
APART = dict(table=(1 << 26, 2 * 4 * 4), indptr=(1 << 27, 3 * 4), kv_len=(1 << 28, 2 * 4))


@pytest.mark.parametrize("name,size", [(k, n) for k, (_, n) in APART.items()] + [("sink", 16 * 4)])
@pytest.mark.parametrize("result", ["out", "lse"])
def test_results_of_chunk_attention_are_apart_from_tables(lib, name, size, result):
    at = {k: p for k, (p, _) in APART.items()}
    at.update(sink=1 << 29, lse=1 << 30, out=1 << 31, ws=1 << 40)
    long = {"out": 3 * 16 * 512 * 2, "lse": 3 * 16 * 4}[result]
    for where in (at[name] - long + 16, at[name], at[name] + (size - 1) // 16 * 16):  # 16-byte aligned
        assert attend(lib, **dict(at, **{result: where})) == INVALID
    if lib.sda_chunk_attention_workspace_size(2, 3, 16, 512, ctypes.byref(ctypes.c_size_t(0))) != OK:
        # (without a GPU nothing is enqueued: what is apart gets as far as the device)
        for where in (at[name] - long, at[name] + (size + 15) // 16 * 16):
            assert attend(lib, **dict(at, **{result: where})) not in (OK, INVALID)


@pytest.mark.parametrize("name", list(APART))
def test_out_of_attention_mass_is_apart_from_tables(lib, name):
    at = {k: p for k, (p, _) in APART.items()}
    at.update(lse=1 << 30, out=1 << 31, ws=1 << 40)
    at_name, size = APART[name]
    for where in (at_name - 2 * 64 * 4 + 4, at_name, at_name + size - 4):
        assert mass(lib, **dict(at, out=where)) == INVALID
    if lib.sda_attention_mass_workspace_size(2, 4, 16, ctypes.byref(ctypes.c_size_t(0))) != OK:
        for where in (at_name - 2 * 64 * 4, at_name + size):
            assert mass(lib, **dict(at, out=where)) not in (OK, INVALID)


def test_evict_slots_counts_in_32_bits(lib):
    """Rows of 2^31 - 2048 columns and 2^24 sequences are the most (every array in a place of its own)."""
    at = dict(scores=1 << 44, table=1 << 45, kv_len=1 << 46, out_scores=1 << 47, out_table=1 << 48, out_len=1 << 49,
              freed=1 << 50, indptr=1 << 51, status=1 << 52, budget=2 ** 31 - 4096, first=0, recent=0)
    for B, stride, refused in ((1, 2 ** 31 - 2047, True), (1, 2 ** 31 - 1, True), (1, 2 ** 31 - 2048, False),
                               (2 ** 24 + 1, 3, True), (2 ** 31 - 1, 0, True), (2 ** 24, 3, False)):
        a = dict(at, B=B, stride=stride, out_stride=stride, capacity=4096)
        if refused:
            assert evict(lib, **a) == INVALID
        elif lib.sda_chunk_attention_workspace_size(2, 3, 16, 512, ctypes.byref(ctypes.c_size_t(0))) != OK:
            assert evict(lib, **a) not in (OK, INVALID)  # (without a GPU: as far as the device)
