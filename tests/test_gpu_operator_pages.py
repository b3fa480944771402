"""Block-table entries outside the page pool: every entry point around the decode
step reports TQ_DEV_PAGE and goes on with page 0 in their place, as the decode does.

Page 0 is nobody's in these caches, so what the calls make of a bad entry is what
they make of a table that names page 0 there."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import assert_close, need_gpu
from tests.operator_helpers import dev, host, make_cache, rows, softmax_rows, values
from tests.test_gpu_evict import heavy, kept_reference
from tests.test_gpu_sparse import attend_reference, bounds_reference, scores_reference, select_reference

pytestmark = pytest.mark.gpu

B, HQ, HKV, N, BLOCK = 2, 8, 2, 500, 64


def paged(tq, torch, D, bits, seed, bad):
    """A filled cache of 4 pages a sequence, none of them page 0; entry (1, 2) is then `bad`, and page 0 holds random rows."""
    c = make_cache(tq, torch, B, HKV, D, N, bits, paged=True, seed=seed, capacity=512)
    pages = np.random.default_rng(seed).permutation(np.arange(1, c.num_pages))[: B * 4].astype(np.int32).reshape(B, 4)
    c.block_table.copy_(torch.from_numpy(pages))
    k = torch.randn((B, HKV, N, D), device="cuda").half()
    tq.tq_quantize_kv_append(c, k, k.flip(2).contiguous(), torch.zeros(B, dtype=torch.int32, device="cuda"))
    for name in ("k_codes", "v_codes", "k_scale", "k_bias", "v_scale", "v_bias"):
        a = getattr(c, name)
        a[0].copy_(a[int(pages[0, 0])])
    torch.cuda.synchronize()
    pages[1, 2] = bad
    c.block_table.copy_(torch.from_numpy(pages))
    return c


class NamesPage0:
    """The cache with page 0 where its table has an entry outside the pool."""

    def __init__(self, c, torch):
        self.__dict__.update(c.__dict__)
        t = c.block_table.clone()
        t[(t < 0) | (t >= c.num_pages)] = 0
        self.block_table, self.paged = t, True
        for name in ("k_codes", "v_codes", "k_scale", "k_bias", "v_scale", "v_bias"):
            setattr(self, name, getattr(c, name))


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_reads(D, bits, bad):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = paged(tq, torch, D, bits, D + bits, bad)
    as0 = NamesPage0(c, torch)
    rng = np.random.default_rng(3)
    q = rng.standard_normal((B, HQ, D)).astype(np.float16)
    lens = dev(torch, np.array([N, N], np.int32))
    scale = 1 / math.sqrt(D)

    def status():
        return torch.zeros(1, dtype=torch.int32, device="cuda")

    st, bounds = status(), tq.block_bounds(c, BLOCK)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    tq.tq_kv_block_bounds(c, bounds, zero, N, block_tokens=BLOCK, status=st)
    assert int(st) == tq.TQ_DEV_PAGE
    want_bounds = bounds_reference(as0, BLOCK, [0, 0], N, np.zeros(tuple(bounds.shape), np.float16))
    assert np.array_equal(bounds.cpu().numpy(), want_bounds)

    st, ws = status(), tq.sparse_workspace(B, HQ, HKV, D, N, 7, BLOCK)
    blocks = torch.zeros((B, HKV, 7), dtype=torch.int32, device="cuda")
    out, _ = tq.tq_sparse_decode(c, bounds, dev(torch, q), lens, N, scale, ws, blocks, block_tokens=BLOCK, status=st)
    want = select_reference(scores_reference(want_bounds, q), [N, N], BLOCK, 7, 1, 1)
    assert np.array_equal(blocks.cpu().numpy(), want)
    assert int(st) == (tq.TQ_DEV_PAGE if any(j in want[1] for j in (4, 5)) else 0)
    assert_close(host(out), attend_reference(as0, q, want, [N, N], BLOCK, scale))

    st, w, wws = status(), torch.zeros((B, HKV, c.capacity), device="cuda"), tq.weights_workspace(B, HQ, HKV, D, N)
    out = tq.tq_sdpa_decode_weights(c, dev(torch, q), lens, N, scale, w, wws, status=st)
    assert int(st) == tq.TQ_DEV_PAGE
    k, v = values(as0, "k"), values(as0, "v")
    for b in range(B):
        for h in range(HKV):
            g = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
            o, p = softmax_rows(q[b, g].astype(np.float64), k[b, h, :N], v[b, h, :N], scale)
            assert_close(host(out)[b, g], o)
            assert np.linalg.norm(host(w)[b, h, :N] - p.sum(0)) <= 1e-5 * np.linalg.norm(p.sum(0))


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_eviction(bad):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    src, dst = paged(tq, torch, 128, 4, 5, bad), paged(tq, torch, 128, 4, 6, 3)
    table = dst.block_table.cpu().numpy()
    table[1, 0] = bad  # page 0 takes its rows
    dst.block_table.copy_(torch.from_numpy(table))
    rng = np.random.default_rng(7)
    w = heavy(rng, (B, HKV, src.capacity))
    keep, recent = 200, 90
    dw, dl = torch.zeros((B, HKV, dst.capacity), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept, st = torch.zeros((B, HKV, keep), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(src, dst, dev(torch, w), dev(torch, np.array([N, N], np.int32)), N, keep, recent, dw, dl, kept, status=st)
    assert int(st) == tq.TQ_DEV_PAGE
    s0, d0 = NamesPage0(src, torch), NamesPage0(dst, torch)
    for b in range(B):
        for h in range(HKV):
            r = kept_reference(w[b, h], N, keep, recent)
            assert np.array_equal(kept.cpu().numpy()[b, h], r)
            for name in ("k_codes", "v_scale"):
                assert np.array_equal(rows(d0, name)[b, h, :keep], rows(s0, name)[b, h, r])
