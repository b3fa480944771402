"""Page keeping at the ends of its ranges."""
import pytest

from tests.gpu_helpers import need_gpu
from tests.test_gpu_pages import i32, pool

pytestmark = pytest.mark.gpu


def test_rows_of_the_largest_cache():
    """A cache of almost 2^31 tokens: all of its rows at once are more than there are pages for, some fit."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    page, per = 384, (2 ** 31 - 1) // 384
    c, refs, held, _, ws = pool(torch, tq, 1, Hkv=1, page=page, pages=3, per=per)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0]), page * per, ws, status=st)
    assert int(st) == tq.TQ_DEV_NO_PAGE and int(held) == 0 and not bool(refs.any()) and bool((c.block_table == -1).all())
    st.zero_()
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0]), 2 * page + 1, ws, status=st)
    assert int(st) == 0 and int(held) == 3 and c.block_table[0, :4].tolist() == [0, 1, 2, -1] and refs.tolist() == [1, 1, 1]
