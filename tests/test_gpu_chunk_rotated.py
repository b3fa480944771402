"""Chunks over rotated caches against fp64, where sequences are cut into runs (whose
merge rotates the outputs back) and where a call has rows of both kinds.

Tolerances as in test_gpu_chunk.py, with the rounding of the rotated query to fp16
beside that of the keys: a score is off by 2^-11 scale sum_d |(Hq)_d K_d| once more, of
the same variance.  Outputs are turned back in fp32 by H, which has entries of
1 / sqrt(D) alone: a bound e becomes e |H|, a variance v becomes v H^2."""
import math

import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache, values
from tests.test_gpu_chunk import attend, check, queries

pytestmark = pytest.mark.gpu


def hadamard(torch, D):
    h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while h.shape[0] < D:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(D)


def reference(torch, cache, q, lens, scale, rotate):
    """fp64 (output, bound of its error, its variance) [B, n, Hq, D]; the query is rotated in 64 bits."""
    k, v = (torch.from_numpy(values(cache, x)).cuda() for x in "kv")
    B, Hq, n, D = q.shape
    G, H, third = Hq // cache.num_kv_heads, hadamard(torch, D), 2.0 ** -22 / 3
    x_all = q.double() @ H if rotate & 1 else q.double()
    roundings = 2 if rotate & 1 else 1  # of a score's terms
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device="cuda")
    bound, var = out.clone(), out.clone()
    for b in range(B):
        L = int(lens[b])
        seen = torch.arange(L, device="cuda") <= torch.arange(n, device="cuda").unsqueeze(1) + (L - n)
        for h in range(cache.num_kv_heads):
            x, kh, vh = x_all[b, h * G:(h + 1) * G], k[b, h, :L], v[b, h, :L]
            p = torch.softmax((torch.einsum("gid,td->git", x, kh) * scale).masked_fill_(~seen, -math.inf), -1)
            o = torch.einsum("git,td->igd", p, vh)
            pe = p * torch.einsum("gid,td->git", x.abs(), kh.abs()) * (roundings * scale * 2 ** -11)
            e = torch.einsum("git,td->igd", pe, vh.abs()) + o.abs() * pe.sum(-1).t().unsqueeze(-1) + torch.einsum("git,td->igd", p, vh.abs()) * 2 ** -10
            pw = p * p * torch.einsum("gid,td->git", x * x, kh * kh) * (roundings * scale * scale * third)
            w = torch.einsum("git,td->igd", pw, vh * vh) + 2 * o.abs() * torch.einsum("git,td->igd", pw, vh.abs()) + o * o * pw.sum(-1).t().unsqueeze(-1)
            w += 2 * torch.einsum("git,td->igd", p * p, vh * vh) * third
            if rotate & 2:
                o, e, w = o @ H, e @ H.abs(), w @ H.square()
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            out[at], bound[at], var[at] = o, 1.05 * (e + o.abs() * 2 ** -11) + 1e-6, w + o * o * third + 1e-12
    return out, bound, var


@pytest.mark.parametrize("rotate", [1, 2, 3])
@pytest.mark.parametrize("D,bits,B,Hkv,G,n,L", [(64, 4, 2, 2, 4, 3, 9000), (128, 4, 2, 2, 8, 3, 9000), (128, 8, 1, 1, 8, 70, 12000), (64, 8, 1, 2, 2, 200, 12000),
                                                (256, 4, 2, 1, 4, 50, 9000),                                          # cut into runs
                                                (128, 4, 4, 2, 8, 1000, 4000), (64, 8, 4, 2, 8, 1000, 2000), (256, 8, 3, 8, 4, 400, 1500)])  # some cut, others whole
def test_rotated_runs(D, bits, B, Hkv, G, n, L, rotate):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens = [L - 501 * b for b in range(B)]
    lens = [max(n, x) for x in lens]
    c = make_cache(tq, torch, B, Hkv, D, L, bits, seed=D + n, flags=rotate)
    q = queries(torch, (B, Hkv * G, n, D), n)
    got = attend(torch, tq, c, q, lens, flags=rotate)
    check(torch, got, reference(torch, c, q, lens, 1 / math.sqrt(D), rotate), [n] * B)
