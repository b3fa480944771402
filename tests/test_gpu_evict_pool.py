"""Eviction between two block tables over one page pool, compared exactly."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache
from tests.test_gpu_evict import ARRAYS, evict_and_check, heavy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4)])
def test_evict_within_one_pool(D, bits):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n = 3, 2, 890
    src = make_cache(tq, torch, B, Hkv, D, n, bits, paged=True, seed=D, capacity=1024)
    free = sorted(set(range(src.num_pages)) - set(src.block_table.cpu().numpy()[:, :7].flatten().tolist()))  # the eighth is unused
    dst = tq.PagedKVCache(B, Hkv, D, 128, src.num_pages, 1, bits=bits)
    dst.buffer = src.buffer
    for a in ARRAYS:
        setattr(dst.struct, a, getattr(src.struct, a))
        setattr(dst, a, getattr(src, a))
    dst.block_table.copy_(torch.from_numpy(np.array(free[:B], np.int32).reshape(B, 1)))
    w = heavy(np.random.default_rng(1), (B, Hkv, src.capacity))
    assert evict_and_check(tq, torch, src, dst, w, [n, 500, 77], n, 100, 40) == 0
