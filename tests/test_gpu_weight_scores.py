"""Attention weights of the decode that accumulates them, for the scores that are
hardest to keep in fp32: keys whose codes an outlier makes small, non-negative
keys, large queries, two rows that share the softmax.

S is the largest attn_scale * sum_d |q_d| (scale * code_d + |bias_d|) of a row: the
magnitude of what a score is the sum of.  A weight's relative error is at most
twice the absolute error of a score (its own, and the rows' in the sum it is
divided by), plus 2^-20 for the exponential, the sums and the division."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import dev, host, rows, values

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]
B, HKV, N = 2, 2, 2048


def weights_and_reference(tq, torch, k, q, bits):
    """(kernel's weights, fp64 weights [B, Hkv, N], S [B, Hkv]) of keys k [B, Hkv, N, D] and queries q [B, Hq, D]."""
    D, G = k.shape[3], q.shape[1] // HKV
    c = tq.KVCache(B, HKV, D, N, bits=bits)
    c.buffer.zero_()
    kt = dev(torch, k.astype(np.float16))
    tq.tq_quantize_kv_append(c, kt, kt.flip(2).contiguous(), torch.zeros(B, dtype=torch.int32, device="cuda"))
    q = q.astype(np.float16)
    w, scale = torch.zeros((B, HKV, N), device="cuda"), 1 / math.sqrt(D)
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    tq.tq_sdpa_decode_weights(c, dev(torch, q), lens, N, scale, w, tq.weights_workspace(B, HKV * G, HKV, D, N), decay=0.0)
    kk, bias = values(c, "k"), np.abs(np.repeat(rows(c, "k_bias").astype(np.float64), 64, -1))
    parts = kk - np.repeat(rows(c, "k_bias").astype(np.float64), 64, -1) + bias
    qd = q.astype(np.float64).reshape(B, HKV, G, D)
    x = qd @ kk.swapaxes(2, 3) * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).sum(2)
    S = (np.abs(qd) @ parts.swapaxes(2, 3) * scale).max((2, 3))
    return host(w), p, S


def small_codes(rng, D, size):
    """Non-negative keys with one outlier in each group of 64, whose channels the query hardly uses."""
    k, q = 0.3 * np.abs(rng.standard_normal((B, HKV, N, D))), size * rng.standard_normal((B, 2 * HKV, D))
    k[..., 5::64] = 60.0
    q[..., 5::64] *= 0.001
    return k, q


@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_weights_of_keys_with_small_codes(D, bits):
    """The contract, 1e-5 over a head's rows (relative L2) where S is at most 64."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    for seed in range(3):
        k, q = small_codes(np.random.default_rng(seed), D, {64: 22.0, 128: 19.0, 256: 14.0}[D])
        got, want, S = weights_and_reference(tq, torch, k, q, bits)
        assert 2 < S.max() <= 64
        assert (np.linalg.norm(got - want, axis=-1) <= 1e-5 * np.linalg.norm(want, axis=-1)).all()


def two_rows(rng, D, size):
    """Two rows whose scores differ by little share nearly all of the weight."""
    k, q = rng.standard_normal((B, HKV, N, D)), size * rng.standard_normal((B, HKV, D))
    k[:, :, 100] = 3 * np.abs(k[:, :, 100]) * np.sign(q)
    k[:, :, 1700] = k[:, :, 100] * (1 + 0.002 / size * rng.standard_normal((B, HKV, D)))
    return k, q


def positive(rng, D, size):
    return np.abs(rng.standard_normal((B, HKV, N, D))), size * np.abs(rng.standard_normal((B, 3 * HKV, D)))


@pytest.mark.parametrize("make,size,least", [(two_rows, 1, 60), (two_rows, 20, 1000), (positive, 10, 60), (positive, 60, 300), (small_codes, 100, 10)])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_weights_of_large_scores(D, bits, make, size, least):
    """A score sums, for each group of 64 channels, four products of 16 terms one after another (each of whose at most 17
    addends is cut below 2^-23 of the largest: 68 * 2^-23 of the magnitudes), the query's sum, and the groups with their scale
    and bias (fewer than 24 roundings, 12 * 2^-23): 80 * 2^-23 S at most, twice that for a weight.  The sums of the weights are
    at most 64 roundings deep here, and with the exponential and the division below 2^-17."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    k, q = make(np.random.default_rng(D + bits), D, float(size))
    got, want, S = weights_and_reference(tq, torch, k, q, bits)
    assert S.max() >= least
    tol = (160 * 2.0 ** -23 * S + 2.0 ** -17)[..., None]
    assert (np.abs(got - want) <= tol * want + 1e-37).all()
    assert np.abs(got.sum(-1) - q.shape[1] // HKV).max() <= 2.0 ** -17 * q.shape[1] // HKV + 160 * 2.0 ** -23 * S.max()


@pytest.mark.parametrize("G,D,bits", [(1, 64, 8), (1, 128, 4), (3, 256, 4), (8, 128, 8)])
def test_heads_whose_every_score_is_minus_infinity_add_nothing(G, D, bits):
    """Keys of minus infinity (a bias of -inf in every group) under queries that are positive in every channel: the softmax has no
    sum, the output is zeros, and the weights are decay times themselves.  One of the two kv heads has such keys, in all rows or
    in the first ones of every run."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(G + D)
    c = tq.KVCache(B, HKV, D, N, bits=bits)
    k = dev(torch, rng.standard_normal((B, HKV, N, D)).astype(np.float16))
    tq.tq_quantize_kv_append(c, k, k.flip(2).contiguous(), torch.zeros(B, dtype=torch.int32, device="cuda"))
    c.k_bias[0, 0] = -math.inf
    c.k_bias[1, 1, :700] = -math.inf
    q = (0.25 + rng.random((B, HKV * G, D))).astype(np.float16)
    old = rng.random((B, HKV, N)).astype(np.float32)
    w, ws = dev(torch, old), tq.weights_workspace(B, HKV * G, HKV, D, N)
    lens, scale = torch.full((B,), N, dtype=torch.int32, device="cuda"), 1 / math.sqrt(D)
    out = host(tq.tq_sdpa_decode_weights(c, dev(torch, q), lens, N, scale, w, ws, decay=0.5)).reshape(B, HKV, G, D)
    got = host(w)
    assert not out[0, 0].any() and np.array_equal(got[0, 0], 0.5 * old[0, 0].astype(np.float64))
    assert np.array_equal(got[1, 1, :700], 0.5 * old[1, 1, :700].astype(np.float64))
    kk = values(c, "k")
    for b, h in ((0, 1), (1, 0), (1, 1)):
        x = q.reshape(B, HKV, G, D)[b, h].astype(np.float64) @ kk[b, h].T * scale
        p = np.exp(x - x.max(-1, keepdims=True))
        want = 0.5 * old[b, h] + (p / p.sum(-1, keepdims=True)).sum(0)
        # (at most 2^-24 for the sum's rounding, the contract's 1e-5 for the weights: S is below 64 in the finite rows)
        assert np.linalg.norm(got[b, h] - want) <= 1e-5 * np.linalg.norm(want)
