"""The turn back (TQ_ROPE_INVERSE) against autograd of the rotary formula in fp64."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import dev

pytestmark = pytest.mark.gpu


def turned(torch, x, angle, pairs):
    """x [B, n, h, D] turned by angle [B, n, rotary / 2], as [B, h, n, D]."""
    half = angle.shape[-1]
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :half], r[..., half:])
    c, s = torch.cos(angle).unsqueeze(2), torch.sin(angle).unsqueeze(2)
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((r, rest), -1).transpose(1, 2)


@pytest.mark.parametrize("D,rotary,sections", [(64, 64, (32,)), (128, 96, (8, 20, 20)), (256, 256, (16, 48, 64))])
@pytest.mark.parametrize("pairs", [False, True])
def test_rope_inverse_is_what_autograd_gives(pairs, D, rotary, sections):
    """The gradient of both rows, for incoming gradients of the outputs.  Rounded once to fp16 (half a step, 2^-11 of the value, or
    2^-25 below the normal numbers); before that, the fraction of a turn (2^-26 turns), its cosine and sine
    (2^-22) and the products and their sum (3 * 2^-24) in fp32: below 6e-7 of the two terms' magnitudes."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(D)
    B, n = 2, 37
    pos = rng.integers(0, 5000, (len(sections), B, n)).astype(np.int32)
    inv = (1e4 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = dev(torch, (pos[axis].transpose(1, 2, 0).astype(np.float64) * inv.astype(np.float64)))
    xs = [dev(torch, rng.standard_normal((B, n, h, D))).requires_grad_() for h in (6, 2)]
    gs = [dev(torch, rng.standard_normal((B, h, n, D)).astype(np.float16)) for h in (6, 2)]
    sum((turned(torch, x, angle, pairs) * g.double()).sum() for x, g in zip(xs, gs)).backward()
    flags = tq.TQ_ROPE_INVERSE | (tq.TQ_ROPE_PAIRS if pairs else 0)
    back = tq.tq_rope_axes(gs[0].transpose(1, 2), gs[1].transpose(1, 2), dev(torch, pos), dev(torch, inv), sections, flags=flags)
    for x, g, y in zip(xs, gs, back):
        want, got = x.grad, y.transpose(1, 2).double()
        size = 2 * g.double().abs().max()
        assert bool(((got - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25 + 6e-7 * size).all())
