"""What the header says of block bounds: a block's score against them lies at most
its keys' fp16 rounding below any q.k of the block, and keys that are no numbers
are left out."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import dev, make_cache, values
from tests.test_gpu_sparse import scores_reference

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]


@pytest.mark.parametrize("n,block", [(700, 64), (33, 32)])  # the second block of the second has one row
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_scores_bound_every_product_but_for_rounding(D, bits, n, block):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, G = 2, 2, 3
    c = make_cache(tq, torch, B, Hkv, D, n, bits, seed=D + n)
    bounds = tq.block_bounds(c, block)
    tq.tq_kv_block_bounds(c, bounds, torch.zeros(B, dtype=torch.int32, device="cuda"), n, block_tokens=block)
    q = np.random.default_rng(n).standard_normal((B, Hkv * G, D)).astype(np.float16)
    score = scores_reference(bounds.cpu().numpy(), q)  # [B, Hkv, blocks]
    k, g = values(c, "k")[:, :, :n], q.reshape(B, Hkv, G, D).astype(np.float64)
    product = np.einsum("bhgd,bhnd->bhgn", g, k).max(2)
    slack = (np.abs(g)[:, :, :, None] * np.maximum(2.0 ** -11 * np.abs(k), 2.0 ** -25)[:, :, None]).sum(-1).max(2)
    of = np.arange(n) // block
    # (the sums here are fp64: 1e-12 of what they add)
    assert (product <= score[:, :, of] + slack + 1e-12 * np.abs(score).max()).all()


@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_keys_that_are_no_numbers_are_left_out(D, bits):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n, block = 1, 2, 320, 64
    c = make_cache(tq, torch, B, Hkv, D, n, bits, seed=D)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    c.k_scale[:, :, 5::9] = float("nan")
    c.k_bias[:, 1, 130:150] = float("nan")
    bounds = tq.block_bounds(c, block)
    tq.tq_kv_block_bounds(c, bounds, zero, n, block_tokens=block)
    with np.errstate(invalid="ignore"):
        k = values(c, "k").astype(np.float16).reshape(B, Hkv, n // block, block, D)
    lost = np.isnan(k)
    assert lost.any() and not lost.all(3).any()
    assert np.array_equal(bounds[..., 0, :].cpu().numpy(), np.where(lost, np.inf, k).min(3).astype(np.float16))
    assert np.array_equal(bounds[..., 1, :].cpu().numpy(), np.where(lost, -np.inf, k).max(3).astype(np.float16))
