"""Refusals of the chunk kernel's diagnostic, on the host (array pointers are
addresses that are never read)."""
import ctypes

import pytest

import int4_kv_cache_gb300 as tq
from int4_kv_cache_gb300 import build as tqbuild
from tests.test_operator_args import ALIGN, CAPACITY, NULL, OK, SHAPE, WORKSPACE, addr, cache


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
