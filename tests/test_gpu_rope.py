"""Rotary positions with several axes against the formula in fp64.

Tolerance, element by element.  The result u = x1 c -+ x2 s is rounded once to
fp16: half a step, 2^-11 |u| (2^-25 where fp16 is subnormal).  Before that, in
fp32: the fraction of a turn, at most 1/2, is rounded to fp32 (2^-26 turns =
9.4e-8 rad); sincospif is within 2 units in the last place of values up to 1
(2^-22 = 2.4e-7); the two products and the sum round by 2^-24 each of at most
|x1| + |x2|.  Together below 6e-7 (|x1| + |x2|); the reference's fp64 angle of
2^31 * inv_freq <= 2^31 adds 2^31 * 2^-53 = 2.4e-7.  So 1e-6 (|x1| + |x2|)."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import dev, host

pytestmark = pytest.mark.gpu


def reference(x, positions, inv_freq, sections, pairs, inverse=False):
    """x [B, n, H, D] -> fp64 [B, H, n, D] and the magnitude |x1| + |x2| each element comes from."""
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = positions.astype(np.float64)[axis].transpose(1, 2, 0) * inv_freq.astype(np.float64)
    c, s = np.cos(angle)[:, :, None], np.sin(angle)[:, :, None] * (-1 if inverse else 1)
    half = len(axis)
    y, mag = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
    i0, i1 = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if pairs else (np.arange(half), np.arange(half, 2 * half))
    a, b = x[..., i0].astype(np.float64), x[..., i1].astype(np.float64)
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    mag[..., i0] = mag[..., i1] = np.abs(a) + np.abs(b)
    return y.transpose(0, 2, 1, 3), mag.transpose(0, 2, 1, 3)


def check(out, want, mag):
    err = np.abs(host(out) - want)
    tol = np.maximum(np.abs(want) * 2.0 ** -11, 2.0 ** -25) + 1e-6 * mag
    assert (err <= tol).all(), float((err - tol).max())


def inputs(rng, axes, B, n, R, far=131072):
    pos = rng.integers(0, far, (axes, B, n)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(0, R, 2) / R)).astype(np.float32)
    return pos, inv


CASES = [
    # B, n, hq, hkv, D, rotary, sections
    (1, 1, 8, 2, 128, 128, (16, 24, 24)), (32, 1, 64, 8, 128, 128, (16, 24, 24)), (3, 257, 7, 1, 64, 64, (32,)),
    (2, 33, 5, 5, 256, 256, (64, 64)), (1, 1000, 8, 4, 256, 96, (10, 20, 18)), (2, 65, 4, 2, 128, 16, (2, 2, 2, 2)),
    (1, 3, 4, 1, 64, 48, (0, 24, 0)), (1, 5000, 4, 1, 64, 64, (8, 12, 12)),
]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("B,n,hq,hkv,D,R,sections", CASES)
def test_rope_matches_the_formula(B, n, hq, hkv, D, R, sections, pairs):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(n + D)
    qkv = rng.standard_normal((B, n, hq + 2 * hkv, D)).astype(np.float16)  # one projection's rows: q and k are strided views
    pos, inv = inputs(rng, len(sections), B, n, R)
    t = dev(torch, qkv)
    q, k = t[:, :, :hq], t[:, :, hq:hq + hkv]
    flags = tq.TQ_ROPE_PAIRS if pairs else 0
    qo, ko = tq.tq_rope_axes(q, k, dev(torch, pos), dev(torch, inv), sections, flags=flags)
    check(qo, *reference(qkv[:, :, :hq], pos, inv, sections, pairs))
    check(ko, *reference(qkv[:, :, hq:hq + hkv], pos, inv, sections, pairs))
    assert np.array_equal(t.cpu().numpy().view(np.uint16), qkv.view(np.uint16))  # the input is only read


@pytest.mark.parametrize("order", ["heads first", "batch last", "broadcast"])
def test_rope_reads_any_stride(order):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(3)
    B, n, h, D = 3, 19, 6, 128
    x = rng.standard_normal((B, n, h, D)).astype(np.float16)
    pos, inv = inputs(rng, 2, B, n, D)
    if order == "heads first":
        t = dev(torch, x.transpose(0, 2, 1, 3)).transpose(1, 2)
    elif order == "batch last":
        t = dev(torch, x.transpose(1, 2, 0, 3)).permute(2, 0, 1, 3)
    else:
        x[:, :, :] = x[:, :, :1]
        t = dev(torch, x[:, :, :1]).expand(B, n, h, D)
    out = tq.tq_rope_axes(t, None, dev(torch, pos), dev(torch, inv), (32, 32))
    check(out, *reference(x, pos, inv, (32, 32), False))


def test_rope_far_and_negative_positions():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(4)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 0, 1, 2 ** 30 + 12345, 10 ** 9 + 7], np.int32).reshape(1, 1, 7)
    inv = np.concatenate([(1e6 ** (-np.arange(31) / 31)), [1.0]]).astype(np.float32)
    x = rng.standard_normal((1, 7, 2, 64)).astype(np.float16)
    out = tq.tq_rope_axes(dev(torch, x), None, dev(torch, pos), dev(torch, inv), (32,))
    check(out, *reference(x, pos, inv, (32,), False))


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_inverse_is_the_gradient(pairs):
    """The rows' gradient for an incoming gradient g is the turn back of g: against autograd of the formula in fp64, against
    differences of it, and within the output's rounding (the formula is linear, so both are exact up to fp64)."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(5)
    B, n, h, D, R, sections = 2, 11, 3, 128, 96, (8, 20, 20)
    x = rng.standard_normal((B, n, h, D)).astype(np.float16)
    g = rng.standard_normal((B, h, n, D)).astype(np.float16)
    pos, inv = inputs(rng, 3, B, n, R)
    flags = tq.TQ_ROPE_INVERSE | (tq.TQ_ROPE_PAIRS if pairs else 0)
    back = tq.tq_rope_axes(dev(torch, g).transpose(1, 2), None, dev(torch, pos), dev(torch, inv), sections, flags=flags)
    check(back, *reference(g.transpose(0, 2, 1, 3), pos, inv, sections, pairs, inverse=True))
    got = host(back).transpose(0, 2, 1, 3)  # [B, n, h, D], as x

    def loss(y):
        return float((reference(y, pos, inv, sections, pairs)[0] * g.astype(np.float64)).sum())

    for _ in range(40):
        i = tuple(rng.integers(0, m) for m in x.shape)
        up, down = x.astype(np.float64).copy(), x.astype(np.float64).copy()
        up[i] += 0.5
        down[i] -= 0.5
        # |got| < 8 rounds by at most 2^-9; the differences cancel sums of ~1e3 in fp64
        assert abs((loss(up) - loss(down)) - got[i]) <= 2.0 ** -11 * max(abs(got[i]), 1e-3) + 1e-5


def test_rope_in_a_graph_and_on_another_stream():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(6)
    x = rng.standard_normal((2, 5, 4, 128)).astype(np.float16)
    pos, inv = inputs(rng, 3, 2, 5, 128)
    t, p, f = dev(torch, x), dev(torch, pos), dev(torch, inv)
    out = torch.empty((2, 4, 5, 128), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tq.tq_rope_axes(t, None, p, f, (16, 24, 24), q_out=out, stream=s)
    s.synchronize()
    check(out, *reference(x, pos, inv, (16, 24, 24), False))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_rope_axes(t, None, p, f, (16, 24, 24), q_out=out)
    x2, pos2 = x[::-1].copy(), pos + 1000
    t.copy_(dev(torch, x2))
    p.copy_(dev(torch, pos2))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(out, *reference(x2, pos2, inv, (16, 24, 24), False))


def test_rope_empty_and_refused():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    inv = torch.ones(64, device="cuda")
    x = torch.zeros((2, 0, 4, 128), dtype=torch.float16, device="cuda")
    assert tq.tq_rope_axes(x, None, torch.zeros((1, 2, 0), dtype=torch.int32, device="cuda"), inv, (64,)).shape == (2, 4, 0, 128)
    x = torch.zeros((2, 3, 4, 128), dtype=torch.float16, device="cuda")
    pos = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        tq.tq_rope_axes(x.float(), None, pos, inv, (64,))
    with pytest.raises(ValueError):
        tq.tq_rope_axes(x, None, pos[:, :1], inv, (64,))
    with pytest.raises(ValueError):
        tq.tq_rope_axes(x.transpose(2, 3), None, pos, inv, (64,))
    with pytest.raises(tq.TQError):
        tq.tq_rope_axes(x, None, pos, inv, (63,))
    with pytest.raises(tq.TQError):  # in place
        tq.tq_rope_axes(x[:, :1], None, pos[:, :, :1].contiguous(), inv, (64,), q_out=x.view(-1)[: 2 * 4 * 128].view(2, 4, 1, 128))
