"""Argument checks of the entry points around the decode step (rotary
positions, block bounds, sparse decode, weights, eviction): every refusal is
reported on the host before anything is launched, so no GPU is needed (array
pointers are addresses that are never read)."""
import ctypes

import pytest

import int4_kv_cache_gb300 as tq
from int4_kv_cache_gb300 import build as tqbuild

OK, NULL, SHAPE, CAPACITY, WORKSPACE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 6, 7
BASE = 1 << 40  # addresses far apart, never read
I32 = ctypes.c_int32


@pytest.fixture(scope="module")
def L():
    tqbuild.build()
    return tq.lib()


def addr(i, off=0):
    return BASE + (i << 36) + off


def cache(slot=1, B=2, Hkv=4, D=128, cap=1024, bits=4):
    c = tq.tq_kv_cache()
    assert tq.lib().tq_kv_cache_carve_ex(ctypes.byref(c), addr(slot), B, Hkv, D, 64, bits, cap) == OK
    return c


def paged(slot=1, B=2, Hkv=4, D=128, pt=128, pages=16, per=8, bits=4):
    c = tq.tq_paged_kv_cache()
    assert tq.lib().tq_paged_kv_cache_carve(ctypes.byref(c), addr(slot), addr(30), B, Hkv, D, 64, bits, pt, pages, per) == OK
    return c


# ------------------------------------------------------------------------ rope
def rope(L, **kw):
    a = dict(qx=addr(1), qo=addr(2), kx=addr(3), ko=addr(4), strides=(1 << 14, 1024, 128), heads=8, positions=addr(5),
             inv_freq=addr(6), axes=3, sections=(16, 24, 24), batch=2, n=16, d=128, rotary=128, flags=0, with_k=True)
    a.update(kw)
    q = tq.tq_rope_rows(a["qx"], a["qo"], *a["strides"], a["heads"])
    k = tq.tq_rope_rows(a["kx"], a["ko"], *a["strides"], 4)
    sec = None if a["sections"] is None else (I32 * len(a["sections"]))(*a["sections"])
    return L.tq_rope_axes(ctypes.byref(q), ctypes.byref(k) if a["with_k"] else None, a["positions"], a["inv_freq"], a["axes"], sec,
                          a["batch"], a["n"], a["d"], a["rotary"], a["flags"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), OK), (dict(n=0, with_k=False), OK),
    (dict(qx=None), NULL), (dict(qo=None), NULL), (dict(kx=None), NULL), (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(sections=None), NULL),
    (dict(batch=0), SHAPE), (dict(n=-1), SHAPE), (dict(axes=0), SHAPE), (dict(heads=0), SHAPE),
    (dict(rotary=8, sections=(1, 1, 2)), SHAPE), (dict(rotary=144, sections=(24, 24, 24)), SHAPE),
    (dict(rotary=120, sections=(20, 20, 20)), SHAPE),
    (dict(sections=(16, 24, 23)), SHAPE), (dict(sections=(-1, 40, 25)), SHAPE),
    (dict(strides=(-8, 1024, 128)), SHAPE),
    (dict(axes=5, sections=(16, 16, 16, 16, 0)), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(flags=4), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED),
    (dict(qx=addr(1, 2)), ALIGN), (dict(ko=addr(4, 8)), ALIGN), (dict(strides=(1 << 14, 1028, 128)), ALIGN),
    (dict(positions=addr(5, 1)), ALIGN),
    (dict(qo=addr(1)), SHAPE), (dict(qo=addr(3, 256)), SHAPE), (dict(ko=addr(2, 4096)), SHAPE),  # outs over an x, over an out
])
def test_rope_refusals(L, kw, want):
    assert rope(L, **kw) == want


# ---------------------------------------------------------------------- bounds
def test_bounds_bytes(L):
    assert L.tq_block_bounds_bytes(2, 4, 128, 1000, 64) == 2 * 4 * 16 * 2 * 128 * 2
    for bad in ((0, 4, 128, 1000, 64), (2, 0, 128, 1000, 64), (2, 4, 96, 1000, 64), (2, 4, 128, 0, 64), (2, 4, 128, 1000, 16),
                (2, 4, 128, 1000, 48)):
        assert L.tq_block_bounds_bytes(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), OK), (dict(c=None), NULL), (dict(start=None), NULL), (dict(bounds=None), NULL), (dict(n=-1), SHAPE),
    (dict(n=1025), CAPACITY), (dict(block=16), UNSUPPORTED), (dict(block=96), UNSUPPORTED), (dict(bounds=addr(3, 8)), ALIGN),
    (dict(start=addr(2, 2)), ALIGN),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_bounds_refusals(L, layout, kw, want):
    c = cache() if layout == "contiguous" else paged()
    fn = L.tq_kv_block_bounds if layout == "contiguous" else L.tq_paged_kv_block_bounds
    a = dict(c=ctypes.byref(c), start=addr(2), bounds=addr(3), n=1, block=64)
    a.update(kw)
    assert fn(a["c"], a["block"], a["start"], a["n"], a["bounds"], None, None) == want


# ---------------------------------------------------------------------- sparse
def select(L, **kw):
    a = dict(bounds=addr(2), q=addr(3), B=2, hq=32, hkv=4, d=128, cap=4096, lens=addr(4), max_len=4096, block=64, n=16, first=1,
             last=1, flags=0, ws=addr(5), nbytes=1 << 30, blocks=addr(6))
    a.update(kw)
    return L.tq_select_blocks(a["bounds"], a["q"], a["B"], a["hq"], a["hkv"], a["d"], a["cap"], a["lens"], a["max_len"], a["block"],
                              a["n"], a["first"], a["last"], a["flags"], a["ws"], a["nbytes"], a["blocks"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(bounds=None), NULL), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(blocks=None), NULL),
    (dict(B=0), SHAPE), (dict(hq=30), SHAPE), (dict(n=0), SHAPE), (dict(first=-1), SHAPE), (dict(last=-1), SHAPE),
    (dict(first=9, last=8), SHAPE), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), SHAPE), (dict(max_len=0), SHAPE),
    (dict(hq=36), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(block=256), UNSUPPORTED), (dict(flags=4), UNSUPPORTED),
    (dict(cap=1 << 22, max_len=32 * 22528 + 1, block=32), UNSUPPORTED),
    (dict(max_len=4097), CAPACITY), (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE),
    (dict(bounds=addr(2, 2)), ALIGN), (dict(q=addr(3, 2)), ALIGN), (dict(ws=addr(5, 16)), ALIGN), (dict(blocks=addr(6, 2)), ALIGN),
])
def test_select_refusals(L, kw, want):
    assert select(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(c=None), NULL), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(blocks=None), NULL), (dict(out=None), NULL),
    (dict(hq=30), SHAPE), (dict(n=0), SHAPE), (dict(n=1 << 25), SHAPE), (dict(max_len=0), SHAPE),
    (dict(max_len=1025), CAPACITY), (dict(hq=36), UNSUPPORTED), (dict(block=16), UNSUPPORTED), (dict(flags=0x100), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=1000), WORKSPACE), (dict(ws=addr(5, 64)), ALIGN), (dict(q=addr(3, 4)), ALIGN),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
@pytest.mark.parametrize("fused", [False, True])
def test_sparse_refusals(L, fused, layout, kw, want):
    c = cache() if layout == "contiguous" else paged()
    a = dict(c=ctypes.byref(c), q=addr(3), hq=32, lens=addr(4), max_len=1024, blocks=addr(6), n=4, block=64, flags=0, ws=addr(5),
             nbytes=1 << 30, out=addr(7))
    a.update(kw)
    pre = "tq_" if layout == "contiguous" else "tq_paged_"
    if fused:
        got = getattr(L, pre + "sparse_decode")(a["c"], addr(2), a["q"], a["hq"], a["lens"], a["max_len"], 0.1, a["block"], a["n"],
                                                1, 1, a["flags"], a["ws"], a["nbytes"], a["blocks"], a["out"], None, None)
    else:
        got = getattr(L, pre + "sdpa_blocks_decode")(a["c"], a["q"], a["hq"], a["lens"], a["max_len"], 0.1, a["blocks"], a["n"],
                                                     a["block"], a["flags"], a["ws"], a["nbytes"], a["out"], None, None)
    assert got == want


def test_sparse_workspace_bytes(L):
    n = L.tq_sparse_workspace_bytes(1, 64, 8, 128, 131072, 64, 64)
    # the exact scores of every block, 8 bytes each, the rotated query, the decode's workspace over the listed rows
    assert n == 8 * 2048 * 8 + 64 * 128 * 2 + tq.tq_sdpa_workspace_bytes(1, 64, 8, 128, 64 * 64)
    for bad in ((0, 64, 8, 128, 4096, 8, 64), (1, 64, 8, 96, 4096, 8, 64), (1, 64, 8, 128, 0, 8, 64), (1, 64, 8, 128, 4096, 0, 64),
                (1, 64, 8, 128, 4096, 8, 65), (1, 64, 8, 128, 4096, 1 << 24, 128)):
        assert L.tq_sparse_workspace_bytes(*bad) == 0


# --------------------------------------------------------------------- weights
@pytest.mark.parametrize("kw,want", [
    (dict(c=None), NULL), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(hq=30), SHAPE), (dict(max_len=0), SHAPE), (dict(decay=float("nan")), SHAPE), (dict(max_len=1025), CAPACITY),
    (dict(hq=36), UNSUPPORTED), (dict(flags=0x100), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nbytes=1000), WORKSPACE),
    (dict(ws=addr(5, 64)), ALIGN), (dict(w=addr(6, 2)), ALIGN),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_weights_refusals(L, layout, kw, want):
    c = cache() if layout == "contiguous" else paged()
    fn = L.tq_sdpa_decode_weights if layout == "contiguous" else L.tq_paged_sdpa_decode_weights
    a = dict(c=ctypes.byref(c), q=addr(3), hq=32, lens=addr(4), max_len=1024, decay=1.0, w=addr(6), flags=0, ws=addr(5), nbytes=1 << 30,
             out=addr(7))
    a.update(kw)
    assert fn(a["c"], a["q"], a["hq"], a["lens"], a["max_len"], 0.1, a["decay"], a["w"], a["flags"], a["ws"], a["nbytes"], a["out"],
              None, None) == want


def test_weights_workspace_bytes(L):
    n = L.tq_weights_workspace_bytes(2, 64, 8, 128, 1000)
    scores = 2 * 64 * 1000 * 4
    assert n == -(-scores // 256) * 256 + tq.tq_sdpa_workspace_bytes(2, 64, 8, 128, 1000)
    assert L.tq_weights_workspace_bytes(0, 64, 8, 128, 1000) == 0


# -------------------------------------------------------------------- eviction
def evict(L, layout, src_, dst_, **kw):
    a = dict(src=ctypes.byref(src_), dst=ctypes.byref(dst_), w=addr(10), lens=addr(11), max_len=1024, keep=200, recent=20, dw=addr(12),
             dl=addr(13), kept=addr(14))
    a.update(kw)
    fn = L.tq_kv_evict if layout == "contiguous" else L.tq_paged_kv_evict
    return fn(a["src"], a["dst"], a["w"], a["lens"], a["max_len"], a["keep"], a["recent"], a["dw"], a["dl"], a["kept"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(src=None), NULL), (dict(dst=None), NULL), (dict(w=None), NULL), (dict(lens=None), NULL), (dict(dw=None), NULL),
    (dict(dl=None), NULL), (dict(kept=None), NULL),
    (dict(keep=0), SHAPE), (dict(recent=-1), SHAPE), (dict(recent=201), SHAPE), (dict(max_len=0), SHAPE),
    (dict(max_len=1025), CAPACITY), (dict(keep=257), CAPACITY), (dict(w=addr(10, 2)), ALIGN), (dict(kept=addr(14, 1)), ALIGN),
    (dict(dw=addr(10)), SHAPE), (dict(dl=addr(11)), SHAPE), (dict(kept=addr(10, 64)), SHAPE), (dict(kept=addr(12, 64)), SHAPE),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_evict_refusals(L, layout, kw, want):
    if layout == "contiguous":
        src, dst = cache(1), cache(2, cap=256)
    else:
        src, dst = paged(1), paged(2, pages=4, per=2)
    assert evict(L, layout, src, dst, **kw) == want


@pytest.mark.parametrize("other", [dict(B=3), dict(Hkv=2), dict(D=64), dict(bits=8)])
def test_evict_refuses_caches_that_differ(L, other):
    assert evict(L, "contiguous", cache(1), cache(2, **{**dict(cap=256), **other})) == SHAPE


def test_evict_refuses_a_cache_into_itself(L):
    src = cache(1)
    assert evict(L, "contiguous", src, src) == SHAPE
    dst = cache(2, cap=256)
    dst.v_codes = src.k_codes + 4096
    assert evict(L, "contiguous", src, dst) == SHAPE


def test_python_checks_come_before_the_library(L):
    import torch

    x = torch.zeros((1, 1, 2, 128), dtype=torch.float16)
    with pytest.raises(ValueError):
        tq.tq_rope_axes(x, None, torch.zeros((1, 1, 1), dtype=torch.int32), torch.ones(64), [64])  # not on the GPU
    with pytest.raises(ValueError):
        tq.sparse_workspace(1, 8, 2, 128, 1024, 4, block_tokens=48)
    with pytest.raises(ValueError):
        tq.weights_workspace(0, 8, 2, 128, 1024)


def test_caches_and_lists_past_the_limits(L):
    """More than 2^30 tokens, more than 2^24 listed blocks, a paged cache into itself."""
    big = cache(1, B=1, Hkv=1, D=64, cap=(1 << 30) + 16)
    small = cache(20, B=1, Hkv=1, D=64, cap=256)
    assert L.tq_kv_block_bounds(ctypes.byref(big), 64, addr(2), 1, addr(3), None, None) == UNSUPPORTED
    assert select(L, B=1, hq=1, hkv=1, d=64, cap=(1 << 30) + 16) == UNSUPPORTED
    assert select(L, n=(1 << 24) + 1) == SHAPE
    assert L.tq_sdpa_decode_weights(ctypes.byref(big), addr(3), 1, addr(4), 1024, 0.1, 1.0, addr(6), 0, addr(5), 1 << 40, addr(7), None,
                                    None) == UNSUPPORTED
    assert evict(L, "contiguous", big, small) == UNSUPPORTED
    src = paged(1)
    assert evict(L, "paged", src, src) == SHAPE
