"""Refusals of the chunk attention and of its diagnostic, on the host (array pointers are
addresses that are never read)."""
import ctypes

import pytest
import torch

import int4_kv_cache_gb300 as tq
from int4_kv_cache_gb300 import build as tqbuild
from tests.test_operator_args import ALIGN, CAPACITY, NULL, OK, SHAPE, WORKSPACE, addr, cache, paged

CUDA = 5


@pytest.fixture(scope="module")
def L():
    tqbuild.build()
    return tq.lib()


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), OK), (dict(c=None), NULL), (dict(x=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL), (dict(status=None), NULL),
    (dict(limit=0), SHAPE), (dict(limit=100001), SHAPE), (dict(copies=-1), SHAPE), (dict(n=-1), SHAPE), (dict(max_len=1025), CAPACITY),
    (dict(ws=None), WORKSPACE), (dict(nbytes=16), WORKSPACE), (dict(status=addr(8, 2)), ALIGN),
])
def test_selftest_refusals(L, kw, want):
    c = cache()
    a = dict(c=ctypes.byref(c), x=addr(3), n=16, lens=addr(4), max_len=1024, limit=100, copies=0, ws=addr(5), nbytes=1 << 34, out=addr(7), status=addr(8))
    a.update(kw)
    rows = ctypes.byref(tq.tq_query_rows(a["x"], 1 << 17, 1 << 12, 128, 32, a["n"]))
    assert L.tq_chunk_timeout_selftest(a["c"], rows, a["lens"], a["max_len"], 0.1, a["limit"], a["copies"], a["ws"], a["nbytes"], a["out"],
                                       a["status"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK),
    (dict(out=addr(1, 4096)), SHAPE), (dict(out=addr(5, 256)), SHAPE), (dict(out=addr(4)), SHAPE), (dict(out=addr(6)), SHAPE), (dict(out=addr(8)), SHAPE),
    (dict(out=addr(3, 1 << 18)), SHAPE), (dict(out=addr(30)), SHAPE),
    (dict(ws=addr(1)), SHAPE), (dict(ws=addr(3, 1 << 16)), SHAPE), (dict(ws=addr(4)), SHAPE), (dict(ws=addr(6)), SHAPE), (dict(ws=addr(8)), SHAPE),
    (dict(ws=addr(30)), SHAPE), (dict(ws=addr(7)), SHAPE),
    (dict(status=addr(1, 64)), SHAPE), (dict(status=addr(3, 128)), SHAPE), (dict(status=addr(4, 4)), SHAPE), (dict(status=addr(6)), SHAPE),
    (dict(status=addr(30, 32)), SHAPE),
    # what lies behind the ends, and lists that may be one
    (dict(out=addr(3, 2 * ((1 << 17) + 31 * (1 << 12) + 15 * 128 + 128))), OK), (dict(q_lens=addr(4)), OK), (dict(q_lens=addr(4, 8)), OK),
    (dict(status=addr(4, 8)), OK), (dict(status=None), OK),
])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_chunk_overlaps(L, layout, kw, want):
    """What a call writes lies apart from everything else.  (Without a GPU an accepted call ends with a CUDA error.)"""
    if want == OK and torch.cuda.is_available():
        pytest.skip("the addresses of an accepted call are not read here")
    c = cache() if layout == "contiguous" else paged()
    if layout == "contiguous" and addr(30) in (kw.get("out"), kw.get("ws")) or layout == "contiguous" and kw.get("status") == addr(30, 32):
        want = OK  # no block table
        if torch.cuda.is_available():
            pytest.skip("the addresses of an accepted call are not read here")
    a = dict(x=addr(3), q_lens=addr(6), lens=addr(4), ws=addr(5), out=addr(7), status=addr(8))
    a.update(kw)
    rows = ctypes.byref(tq.tq_query_rows(a["x"], 1 << 17, 1 << 12, 128, 32, 16))
    fn = L.tq_sdpa_chunk if layout == "contiguous" else L.tq_paged_sdpa_chunk
    got = fn(ctypes.byref(c), rows, a["q_lens"], a["lens"], 1024, 0.1, 0, 0, a["ws"], 1 << 34, a["out"], a["status"], None)
    assert got == (CUDA if want == OK else want)
