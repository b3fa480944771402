"""Chunk attention where its arithmetic is at an edge.  Tolerances as in
test_gpu_chunk.py where nothing else is said."""
import math

import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache, values
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


def steps_of_weight(torch, tq, D, bits, L, n, G, keys, seed):
    """(output, fp64 output, fp64 sum_t p_t |V_t|, max_t p_t sum_t |V_t|) of rows that all have the weights
    2^keys[t]: keys that hold multiples of 1/16 and values of 1/8 are exact in fp16, queries select a channel."""
    c = tq.KVCache(1, 1, D, L, bits=bits)
    c.buffer.zero_()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c.v_codes.copy_(torch.randint(0, 256, c.v_codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.v_scale.fill_(1 / 8)
    c.v_bias.fill_(0.5)
    c.k_bias[0, 0] = keys.half().unsqueeze(-1)
    none = keys == keys.max()  # what holds most of the weight has nothing to add
    for a in (c.v_scale, c.v_bias):
        a[0, 0, none] = 0
    q = torch.zeros((1, G, n, D), dtype=torch.float16, device="cuda")
    q[..., 1] = 1
    got = attend(torch, tq, c, q, [L], full=True, scale=math.log(2))
    v = torch.from_numpy(values(c, "v")).cuda()[0, 0]
    p = torch.softmax(keys.double() * math.log(2), 0)
    return got[0], p @ v, p @ v.abs(), float(p.max()) * v.abs().sum(0)


@pytest.mark.parametrize("below", [13, 18, 22, 25, 28])
@pytest.mark.parametrize("at", [0, 2047])
@pytest.mark.parametrize("n,G", [(4864, 8), (5, 4), (300, 1)])  # uncut runs of keys, runs of one and of two row tiles
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 4), (128, 8), (256, 4)])
def test_a_key_that_holds_most_of_the_weight(D, bits, n, G, at, below):
    """The others' weights, 2^-below of its own, make up the output.  Off by half a step of fp16 of the output, of each
    weight (2^-11), and half a subnormal one of the weights below 2^-21 (2^-32 of the largest); fp32 scores and
    exponents up to 2^5 are off by 2^-19, exponentials of them by 2^-18 in numerator and sum; the products' sums take
    256 steps, each of which may lose a unit of fp32's last place, 2^-23 of the sum so far, from 17 terms: 2^-12."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    if n > 4000 and D == 256:
        n //= 2
    L = 4096
    jitter = torch.randint(0, 16, (L,), generator=torch.Generator().manual_seed(below), dtype=torch.int32).cuda() / 16
    keys = -(below + jitter)
    keys[at] = 0
    got, want, weight, total = steps_of_weight(torch, tq, D, bits, L, n, G, keys, below)
    bound = want.abs() * 2 ** -11 + weight * (2 ** -11 + 2 ** -12 + 2 ** -16) + total * 2.0 ** -32
    assert float(((got.double() - want).abs() / bound).max()) <= 1.0


@pytest.mark.parametrize("up", [7.9375, 8, 8.0625, 15])
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_maxima_that_grow(D, bits, up):
    """Later keys above the first ones by as much as is left alone, or a little more: weights up to 2^15."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    L = 2048
    keys = torch.zeros(L, device="cuda")
    keys[1000:] = up
    keys[1500] = up + 1 / 16
    got, want, weight, total = steps_of_weight(torch, tq, D, bits, L, 70, 4, keys, 1)
    assert bool(torch.isfinite(got).all())
    bound = want.abs() * 2 ** -11 + weight * (2 ** -11 + 2 ** -12 + 2 ** -16) + total * 2.0 ** -32
    assert float(((got.double() - want).abs() / bound).max()) <= 1.0
