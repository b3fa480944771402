"""Argument checks of the entry points for several query rows and for pages: every
refusal is reported on the host before anything is launched, so no GPU is needed
(array pointers are addresses that are never read)."""
import ctypes

import pytest

import int4_kv_cache_gb300 as tq
from int4_kv_cache_gb300 import build as tqbuild
from tests.test_operator_args import ALIGN, CAPACITY, NULL, OK, SHAPE, UNSUPPORTED, WORKSPACE, addr, cache, paged


@pytest.fixture(scope="module")
def L():
    tqbuild.build()
    return tq.lib()


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), OK), (dict(n=0, ws=None), OK),
    (dict(c=None), NULL), (dict(x=None), NULL), (dict(rows=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(heads=30), SHAPE), (dict(heads=0), SHAPE), (dict(n=-1), SHAPE), (dict(strides=(-8, 8, 8)), SHAPE), (dict(strides=(0, 0, -8)), SHAPE),
    (dict(max_len=0), SHAPE), (dict(window=-1), SHAPE), (dict(n=(1 << 28) // 32 + 1), SHAPE), (dict(out=addr(3, 64)), SHAPE),
    (dict(x=addr(7, 4096)), SHAPE), (dict(max_len=1025), CAPACITY),
    (dict(heads=36), UNSUPPORTED), (dict(flags=0x100), UNSUPPORTED), (dict(flags=4), UNSUPPORTED), (dict(flags=0x200, window=5), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=16), WORKSPACE), (dict(ws=addr(5, 64)), ALIGN), (dict(x=addr(3, 8)), ALIGN),
    (dict(out=addr(7, 2)), ALIGN), (dict(strides=(4, 128, 128)), ALIGN), (dict(lens=addr(4, 2)), ALIGN), (dict(q_lens=addr(6, 1)), ALIGN),
    (dict(status=addr(8, 2)), ALIGN),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_chunk_refusals(L, layout, kw, want):
    c = cache() if layout == "contiguous" else paged()
    a = dict(c=ctypes.byref(c), x=addr(3), heads=32, n=16, strides=(1 << 17, 1 << 12, 128), lens=addr(4), q_lens=addr(6), max_len=1024, window=0, flags=0,
             ws=addr(5), nbytes=1 << 34, out=addr(7), status=addr(8))
    a.update(kw)
    rows = ctypes.byref(tq.tq_query_rows(a["x"], *a["strides"], a["heads"], a["n"])) if a.get("rows", 0) is not None else None
    fn = L.tq_sdpa_chunk if layout == "contiguous" else L.tq_paged_sdpa_chunk
    assert fn(a["c"], rows, a["q_lens"], a["lens"], a["max_len"], 0.1, a["window"], a["flags"], a["ws"], a["nbytes"], a["out"], a["status"], None) == want


def test_chunk_workspace_bytes(L):
    assert L.tq_chunk_workspace_bytes(1, 64, 8, 128, 8, 131072) > 0
    for bad in ((0, 64, 8, 128, 8, 1024), (1, 63, 8, 128, 8, 1024), (1, 72, 8, 128, 8, 1024), (1, 64, 8, 96, 8, 1024), (1, 64, 8, 128, 0, 1024),
                (1, 64, 8, 128, 8, 0), (1, 64, 8, 128, 1 << 23, 1024), (65536, 64, 8, 128, 1, 1024), (1, 64, 8, 128, 8, (1 << 30) + 1)):
        assert L.tq_chunk_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("sizes", [(1, 64, 8, 128, 8, 131072), (32, 64, 8, 128, 256, 8192), (1, 1, 1, 64, 1, 16), (16, 16, 16, 256, 448, 1500)])
def test_chunk_workspace_grows(L, sizes):
    """A workspace serves fewer rows, shorter sequences and smaller batches of the same heads."""
    b, hq, hkv, d, n, s = sizes
    full = L.tq_chunk_workspace_bytes(*sizes)
    for fewer in ((b, hq, hkv, d, max(1, n // 3), s), (b, hq, hkv, d, 1, s), (b, hq, hkv, d, n, max(1, s // 5)), (1, hq, hkv, d, n, s),
                  (max(1, b // 2), hq, hkv, d, max(1, n - 1), 1)):
        assert 0 < L.tq_chunk_workspace_bytes(*fewer) <= full


def pages_call(L, fn, **kw):
    c = paged()
    a = dict(c=ctypes.byref(c), refs=addr(2), held=addr(3), lens=addr(4), src=addr(5), ws=addr(6), nbytes=1 << 30, status=addr(7), n=1,
             table=addr(8), refs_out=addr(9), n_live=addr(10), moved=addr(11))
    a.update(kw)
    tail = (a["ws"], a["nbytes"], a["status"], None)
    if fn == "fork":
        return L.tq_pages_fork(a["c"], a["refs"], a["held"], a["lens"], a["src"], *tail)
    if fn == "reserve":
        return L.tq_pages_reserve(a["c"], a["refs"], a["held"], a["src"], a["n"], *tail)
    return L.tq_pages_compact(a["c"], a["refs"], a["held"], a["table"], a["refs_out"], a["n_live"], a["moved"], *tail)


@pytest.mark.parametrize("kw,want", [
    (dict(c=None), NULL), (dict(refs=None), NULL), (dict(held=None), NULL), (dict(ws=None), WORKSPACE), (dict(nbytes=1000), WORKSPACE),
    (dict(ws=addr(6, 16)), ALIGN), (dict(refs=addr(2, 2)), ALIGN), (dict(held=addr(3, 1)), ALIGN), (dict(status=addr(7, 2)), ALIGN),
    (dict(ws=addr(30)), SHAPE),       # over the block table
    (dict(ws=addr(1, 4096)), SHAPE),  # over the cache
])
@pytest.mark.parametrize("fn", ["fork", "reserve", "compact"])
def test_pages_refusals(L, fn, kw, want):
    assert pages_call(L, fn, **kw) == want


@pytest.mark.parametrize("fn,kw,want", [
    ("fork", dict(src=None), NULL), ("fork", dict(src=addr(4)), SHAPE), ("fork", dict(lens=addr(3, 4)), SHAPE), ("fork", dict(src=addr(30, 60)), SHAPE),
    ("fork", dict(lens=addr(4, 2)), ALIGN), ("fork", dict(src=addr(5, 2)), ALIGN), ("fork", dict(refs=addr(3)), SHAPE), ("fork", dict(status=addr(2, 60)), SHAPE),
    ("fork", dict(lens=addr(1)), SHAPE),
    ("reserve", dict(n=0), OK), ("reserve", dict(n=-1), SHAPE), ("reserve", dict(n=1025), CAPACITY), ("reserve", dict(src=None), NULL),
    ("reserve", dict(src=addr(3)), SHAPE), ("reserve", dict(src=addr(1)), SHAPE), ("reserve", dict(src=addr(5, 2)), ALIGN),
    ("compact", dict(table=None), NULL), ("compact", dict(refs_out=None), NULL), ("compact", dict(n_live=None), NULL),
    ("compact", dict(table=addr(30, 4)), SHAPE), ("compact", dict(refs_out=addr(2, 4)), SHAPE), ("compact", dict(refs_out=addr(8)), SHAPE),
    ("compact", dict(moved=addr(2)), SHAPE), ("compact", dict(n_live=addr(9, 4)), SHAPE), ("compact", dict(table=addr(2)), SHAPE),
    ("compact", dict(refs_out=addr(30)), SHAPE), ("compact", dict(table=addr(1)), SHAPE), ("compact", dict(moved=addr(11, 2)), ALIGN),
    ("compact", dict(table=addr(8, 2)), ALIGN), ("compact", dict(n_live=addr(3)), SHAPE),
])
def test_pages_refusals_of_each(L, fn, kw, want):
    assert pages_call(L, fn, **kw) == want


def test_pages_workspace_bytes(L):
    assert L.tq_pages_workspace_bytes(32, 4096, 128) > 4096 * 8 + 32 * 128 * 4
    for bad in ((0, 16, 8), (2, 0, 8), (2, 16, 0), (1 << 16, 16, 1 << 15)):
        assert L.tq_pages_workspace_bytes(*bad) == 0
