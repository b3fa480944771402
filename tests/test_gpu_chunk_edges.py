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


def test_windows_of_any_size():
    """A window that 32 bits do not hold is none, not what is left of it."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 2, 128, 700, seed=5)
    q = queries(torch, (1, 8, 90, 128), 6)
    want = attend(torch, tq, c, q, [700])
    for window in (2 ** 31, 2 ** 32 + 10, 2 ** 63 - 1):
        assert torch.equal(attend(torch, tq, c, q, [700], window=window), want)


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
    keys = keys.half()  # (steps of 1/16 up to 128, of 1/4 up to 512)
    c.k_bias[0, 0] = keys.unsqueeze(-1)
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


# A chain of an accumulator is 8,192 keys, 512 steps of 17 terms (16 products and the sum so far), each cut off by less
# than a unit of fp32's last place, 2^-23 of the sum so far, which is half the whole one on average.
CHAIN = 512 * 17 * 2.0 ** -23 / 2


@pytest.mark.parametrize("D,bits,Hkv,n,G,L", [(128, 4, 1, 4864, 8, 262144), (64, 8, 1, 4864, 8, 262144), (256, 4, 1, 2432, 8, 262144),  # uncut
                                              (128, 8, 1, 3200, 8, 65536), (256, 8, 1, 1600, 8, 65536),  # cut into runs that are longer than a chain
                                              (64, 4, 160, 3, 8, 65536), (128, 4, 160, 1, 8, 65536)])    # one row tile, keys in turn to two accumulators
def test_long_runs(D, bits, Hkv, n, G, L):
    """Values around 1 under weights of many sizes: nothing adds up along a sequence.  (Products are exact in fp16 but for
    the weights; every row is the same one.)"""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = tq.KVCache(1, Hkv, D, L, bits=bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(L + D)
    for a in (c.k_codes, c.v_codes):
        a.copy_(torch.randint(0, 256, a[:, :1].shape, generator=g, device="cuda", dtype=torch.uint8).expand_as(a))
    step = 1 / 16 if bits == 4 else 1 / 256
    for a, x in ((c.k_scale, 4 * step), (c.k_bias, -2.0), (c.v_scale, step), (c.v_bias, 0.5)):
        a.fill_(x)
    q = (torch.randn((1, 1, 1, D), generator=g, device="cuda").half() * 0.3).expand(1, Hkv * G, n, D)
    rows = [n] if n == 1 else None  # (single rows as a chunk's)
    got = attend(torch, tq, c, q, [L], rows, full=True)[0].double()

    def exact(codes, scale, bias):
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2) if bits == 4 else codes
        return codes.double() * scale + bias

    p = torch.softmax(exact(c.k_codes[0, 0], 4 * step, -2.0) @ q[0, 0, 0].double() / math.sqrt(D), 0)
    want = p @ exact(c.v_codes[0, 0], step, 0.5)  # positive values: also the weights' sum of them
    assert float(((got - want).abs() / want).max()) <= 2 * 2 ** -11 + CHAIN + 2 ** -16
    # Signed, over all channels: half of what is cut off, and what is left of 64 or more roundings of the output, even
    # over half a step either way (six times 2^-11 / sqrt(3 * 64)).
    assert abs(float((got - want).mean() / want.mean())) <= CHAIN / 2 + 6 * 2 ** -11 / math.sqrt(3 * 64)


@pytest.mark.parametrize("rise", [30, -30, 0.5, 90, 400])
@pytest.mark.parametrize("D,bits,n,G", [(64, 8, 4864, 8), (128, 4, 4864, 8), (256, 4, 2432, 8), (128, 4, 3200, 8), (128, 4, 1, 4)])
def test_long_runs_of_growing_weights(D, bits, n, G, rise):
    """Weights that grow, or fall, over five chains, also by more than fp32 holds."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    L = 40960
    keys = (torch.arange(L, device="cuda") * (16 * rise) / L).floor() / 16
    got, want, weight, total = steps_of_weight(torch, tq, D, bits, L, n, G, keys, n)
    bound = want.abs() * 2 ** -11 + weight * (2 ** -11 + CHAIN + 2 ** -16) + total * 2.0 ** -32
    assert float(((got.double() - want).abs() / bound).max()) <= 1.0


@pytest.mark.parametrize("D,n", [(64, 4864), (128, 4864), (256, 2432)])
def test_workspace_of_long_runs_holds_anything(D, n):
    """What accumulators are emptied into is written before it is read."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    L = 30000
    c = make_cache(tq, torch, 1, 1, D, L, seed=n)
    q = queries(torch, (1, 8, n, D), n)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    ws = tq.chunk_workspace(1, 8, 1, D, n, L)
    outs = []
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        outs.append(tq.tq_sdpa_chunk(c, q, lens, L, 0.1, ws))
    assert bool(torch.isfinite(outs[0]).all()) and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check(torch, outs[0][:, -64:], reference(torch, c, q[:, :, -64:], [L], [64], 0.1), [64])
