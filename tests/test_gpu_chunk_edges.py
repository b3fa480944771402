"""Chunk attention where its arithmetic is at an edge.  Tolerances as in
test_gpu_chunk.py where nothing else is said."""
import math

import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache
from tests.test_gpu_chunk import attend, check, queries, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 701, 700])
@pytest.mark.parametrize("D,bits,paged", [(64, 8, True), (128, 4, False), (256, 4, False)])
def test_wide_windows_over_short_sequences(D, bits, paged, window):
    """A window past the length is none, also where a sequence has fewer tokens than rows."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens, n = [4, 30, 0, 1, 700], 90
    c = make_cache(tq, torch, 5, 2, D, 700, bits, paged, seed=5, capacity=768)
    q = queries(torch, (5, 8, n, D), 6)
    want = attend(torch, tq, c, q, lens)
    check(torch, want, reference(torch, c, q, lens, [n] * 5, 1 / math.sqrt(D)), [n] * 5)
    assert torch.equal(attend(torch, tq, c, q, lens, window=window), want)
