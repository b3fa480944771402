"""Eviction refuses calls whose written arrays overlap what it reads or each
other; on the host, before anything is launched (addresses are never read)."""
import ctypes

import pytest

from tests.test_operator_args import SHAPE, L, addr, cache, evict, paged  # noqa: F401 (L: a fixture)

ARRAYS = ["k_codes", "v_codes", "k_scale", "k_bias", "v_scale", "v_bias"]


def pair(layout):
    if layout == "contiguous":
        return cache(1), cache(2, cap=256)
    dst = paged(2, pages=4, per=2)
    dst.block_table = addr(31)
    return paged(1), dst


def size(c, name):
    """Bytes of a cache array."""
    rows = c.batch * c.num_kv_heads * c.capacity if hasattr(c, "capacity") else c.num_pages * c.num_kv_heads * c.page_tokens
    return rows * (c.head_dim * c.bits // 8 if "codes" in name else c.head_dim // 64 * 2)


@pytest.mark.parametrize("name", ARRAYS)
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_outputs_inside_the_cache_arrays(L, layout, name):  # noqa: F811
    for what in ("dw", "dl", "kept"):
        for which in (0, 1):
            both = pair(layout)
            at, n = getattr(both[which], name), size(both[which], name)
            assert evict(L, layout, *both, **{what: at + 64}) == SHAPE
            assert evict(L, layout, *both, **{what: at + n - 4}) == SHAPE  # its last bytes


@pytest.mark.parametrize("name", ARRAYS)
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_destination_arrays_over_what_is_read(L, layout, name):  # noqa: F811
    src, dst = pair(layout)
    for at in (addr(10, 256), addr(11), getattr(src, name) + 256, src.v_bias, src.k_codes):
        src, dst = pair(layout)
        setattr(dst, name, at)
        assert evict(L, layout, src, dst) == SHAPE


def test_block_tables(L):  # noqa: F811
    for what in ("dw", "dl", "kept"):
        src, dst = pair("paged")
        assert evict(L, "paged", src, dst, **{what: src.block_table + 8}) == SHAPE
        assert evict(L, "paged", src, dst, **{what: dst.block_table + 8}) == SHAPE
    src, dst = pair("paged")
    dst.v_scale = src.block_table & ~15
    assert evict(L, "paged", src, dst) == SHAPE


def test_pools_that_share_some_of_their_memory(L):  # noqa: F811
    """One pool is one pool in all six arrays and in the pages' size; anything else that overlaps is refused."""
    src = paged(1)
    for name in ARRAYS:
        dst = paged(1, pages=8, per=2)  # as carved: the arrays behind the first begin elsewhere
        dst.block_table = addr(31)
        assert evict(L, "paged", src, dst) == SHAPE
        dst = paged(2, pages=4, per=2)
        dst.block_table = addr(31)
        setattr(dst, name, getattr(src, name))
        assert evict(L, "paged", src, dst) == SHAPE
    dst = paged(1, pt=256, pages=8, per=2)
    dst.block_table = addr(31)
    assert [getattr(dst, n) for n in ARRAYS] == [getattr(src, n) for n in ARRAYS]
    assert evict(L, "paged", src, dst) == SHAPE
    assert evict(L, "paged", src, src) == SHAPE


def test_destination_arrays_over_each_other(L):  # noqa: F811
    for layout in ("contiguous", "paged"):
        src, dst = pair(layout)
        dst.v_codes = dst.k_codes
        assert evict(L, layout, src, dst) == SHAPE
        src, dst = pair(layout)
        dst.v_bias = addr(12, 16)
        assert evict(L, layout, src, dst) == SHAPE
