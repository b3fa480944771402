"""Attention of several query rows over the cache against fp64.

Tolerances.  A cached value enters rounded to fp16, off by half a step, 2^-11 of it.
Of the keys that moves the score of token t by e_t = 2^-11 scale sum_d |q_d K_td| at
most, and through d p_t = p_t (d s_t - sum_u p_u d s_u) the output by at most
sum_t p_t e_t |V_t| + |o| sum_t p_t e_t.  The values' rounding and that of the softmax
weights (2^-11 each) add 2^-10 sum_t p_t |V_t|, the output's own 2^-11 |o|; sums in
fp32 and what falls below fp16's normal range some 1e-6.  Each value is held to the sum of
these, with 5 % for the terms of second order (e_t reaches 0.03).

All rows together are held to twice the root of the sum of the variances: a rounding is
even over its step, of variance (half a step)^2 / 3, and independent of the others, so
a score's variance is at most scale^2 sum_d (q_d K_td)^2 2^-22 / 3 =: w_t, an output's
sum_t p_t^2 w_t (|V_t| + |o|)^2 + (2 sum_t p_t^2 V_t^2 + o^2) 2^-22 / 3.  (Rows share
keys and values, which leaves the sum's expectation as it is.)"""
import math

import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache, values

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]


def reference(torch, cache, q, lens, rows, scale, window=0, full=False):
    """fp64 (output, bound of its error, its variance) [B, n, Hq, D] (rows behind rows[b]: NaN)."""
    k, v = (torch.from_numpy(values(cache, x)).cuda() for x in "kv")
    B, Hq, n, D = q.shape
    G = Hq // cache.num_kv_heads
    out = torch.full((B, n, Hq, D), math.nan, dtype=torch.float64, device="cuda")
    bound, var = out.clone(), out.clone()
    for b in range(B):
        L, r = int(lens[b]), int(rows[b])
        t, pos = torch.arange(L, device="cuda"), torch.arange(r, device="cuda") + (L - r)
        seen = torch.ones((r, L), dtype=torch.bool, device="cuda")
        if not full:
            seen = t <= pos.unsqueeze(1)
            if window:
                seen &= t > pos.unsqueeze(1) - window
        for h in range(cache.num_kv_heads):
            x, kh, vh = q[b, h * G:(h + 1) * G, :r].double(), k[b, h, :L], v[b, h, :L]
            s = torch.einsum("gid,td->git", x, kh) * scale
            s.masked_fill_(~seen, -math.inf)
            p = torch.softmax(s, -1) if L else s
            p = torch.where(seen.any(-1).view(1, -1, 1), p, torch.zeros_like(p))
            o = torch.einsum("git,td->igd", p, vh)
            pe = p * torch.einsum("gid,td->git", x.abs(), kh.abs()) * (abs(scale) * 2 ** -11)
            e = torch.einsum("git,td->igd", pe, vh.abs()) + o.abs() * pe.sum(-1).t().unsqueeze(-1)
            e += torch.einsum("git,td->igd", p, vh.abs()) * 2 ** -10 + o.abs() * 2 ** -11
            third = 2.0 ** -22 / 3
            pw = p * p * torch.einsum("gid,td->git", x * x, kh * kh) * (scale * scale * third)
            w = torch.einsum("git,td->igd", pw, vh * vh) + 2 * o.abs() * torch.einsum("git,td->igd", pw, vh.abs()) + o * o * pw.sum(-1).t().unsqueeze(-1)
            w += (2 * torch.einsum("git,td->igd", p * p, vh * vh) + o * o) * third
            at = (b, slice(0, r), slice(h * G, (h + 1) * G))
            out[at], bound[at], var[at] = o, 1.05 * e + 1e-6, w + 1e-12
    return out, bound, var


def check(torch, got, ref, rows):
    want, bound, var = ref
    for b, r in enumerate(rows):
        g, w = got[b, :r].double(), want[b, :r]
        assert bool(torch.isfinite(g).all())
        over = (g - w).abs() / bound[b, :r]
        assert r == 0 or float(over.max()) <= 1.0, f"sequence {b}: {float(over.max()):.2f} of the bound"
    err = sum(float((got[b, :r].double() - want[b, :r]).square().sum()) for b, r in enumerate(rows))
    expected = sum(float(var[b, :r].sum()) for b, r in enumerate(rows))
    assert err <= 4 * expected, f"{math.sqrt(err / expected):.2f} times the expected error"


def attend(torch, tq, cache, q, lens, rows=None, window=0, full=False, flags=0, scale=None, max_len=None, out=None, status=None):
    B, Hq, n, D = q.shape
    most = max_len or max(1, int(max(lens)))
    ws = tq.chunk_workspace(B, Hq, cache.num_kv_heads, D, n, most)
    ql = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    return tq.tq_sdpa_chunk(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), most, scale or 1 / math.sqrt(D), ws, out=out,
                            q_lens=ql, window=window, flags=flags | (tq.TQ_CHUNK_FULL if full else 0), status=status)


def queries(torch, shape, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float16)).cuda()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_ragged_chunks(D, bits, G, paged):
    """Lengths and rows from none to more rows than the sequence has tokens; what lies behind is left alone."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    Hkv, n, L = 2, 150, 700
    lens, rows = [700, 0, 1, 333, 128, 60, 512, 385], [150, 0, 1, 17, 128, 150, 0, 129]
    c = make_cache(tq, torch, len(lens), Hkv, D, L, bits, paged, seed=D + G, capacity=768)
    q = queries(torch, (len(lens), Hkv * G, n, D), G)
    out = torch.full((len(lens), n, Hkv * G, D), 7.0, dtype=torch.float16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    attend(torch, tq, c, q, lens, rows, out=out, status=st)
    check(torch, out, reference(torch, c, q, lens, rows, 1 / math.sqrt(D)), rows)
    for b, r in enumerate(rows):
        assert bool((out[b, r:] == 7.0).all())
    assert not bool(out[5, :90].any())  # rows before the first token
    assert int(st) == 0


@pytest.mark.parametrize("n", [1, 2, 5, 16, 17, 31, 64, 129])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8), (128, 1), (128, 5), (256, 2), (256, 7)])
def test_few_rows(D, G, n):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens = [2500, 131, 129]
    c = make_cache(tq, torch, 3, 2, D, 2500, 4, False, seed=n)
    q = queries(torch, (3, 2 * G, n, D), n)
    got = attend(torch, tq, c, q, lens)
    assert got.shape == (3, n, 2 * G, D)
    check(torch, got, reference(torch, c, q, lens, [n] * 3, 1 / math.sqrt(D)), [n] * 3)


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("D,bits,paged", [(64, 8, False), (128, 4, True), (256, 4, False)])
def test_window(D, bits, paged, window):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens, rows = [900, 400, 33], [200, 400, 40]
    c = make_cache(tq, torch, 3, 2, D, 900, bits, paged, seed=window, capacity=1024)
    q = queries(torch, (3, 6, 400, D), window)
    got = attend(torch, tq, c, q, lens, rows, window=window)
    check(torch, got, reference(torch, c, q, lens, rows, 1 / math.sqrt(D), window), rows)


@pytest.mark.parametrize("n", [1, 77, 300])
@pytest.mark.parametrize("D,bits,G,paged", [(64, 8, 1, False), (64, 4, 4, True), (128, 4, 2, False), (256, 8, 1, False)])
def test_cross(D, bits, G, paged, n):
    """Every row over the whole sequence, longer and shorter than the rows, and none."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens = [1500, 40, 0, 1, 257]
    c = make_cache(tq, torch, 5, 3, D, 1500, bits, paged, seed=n, capacity=1536)
    q = queries(torch, (5, 3 * G, n, D), n)
    rows = [n, max(1, n // 2), n, n, n]
    got = attend(torch, tq, c, q, lens, rows, full=True)
    check(torch, got, reference(torch, c, q, lens, rows, 1 / math.sqrt(D), full=True), rows)


@pytest.mark.parametrize("n", [3, 140])
@pytest.mark.parametrize("rotate", [1, 2, 3])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_rotated(D, bits, rotate, n):
    """A rotated cache gives what the unrotated rows of the same codes would."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens = [600, 300]
    c = make_cache(tq, torch, 2, 2, D, 600, bits, False, seed=D, flags=rotate)
    q = queries(torch, (2, 8, n, D), D)
    got = attend(torch, tq, c, q, lens, flags=rotate)
    qr = tq.tq_hadamard_rotate(q) if rotate & 1 else q
    want = reference(torch, c, qr, lens, [n] * 2, 1 / math.sqrt(D))
    if rotate & 2:
        h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
        while h.shape[0] < D:
            h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
        h /= math.sqrt(D)
        o = want[0] @ h
        want = (o, want[1] @ h.abs() + o.abs() * 2 ** -11, want[2] @ h.square() + o.square() * (2 ** -22 / 3))
    check(torch, got, want, [n] * 2)


def test_strided_query():
    """Rows of a fused projection, heads and tokens in either order."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 2, 2, 128, 300, seed=1)
    big = queries(torch, (2, 40, 12, 128), 3)  # [B, n, heads, D]
    q = big[:, :, 2:10].transpose(1, 2)
    got = attend(torch, tq, c, q, [300, 200])
    assert torch.equal(got, attend(torch, tq, c, q.contiguous(), [300, 200]))
    # single rows: contiguous ones take the decode kernel, others the tiles (not the same bits)
    one = big[:, :1, :8].transpose(1, 2)
    want = reference(torch, c, one, [300, 200], [1, 1], 1 / math.sqrt(128))
    for q in (one, one.contiguous()):
        check(torch, attend(torch, tq, c, q, [300, 200]), want, [1, 1])


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 3.0])
def test_scales(scale):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 2, 64, 400, seed=2, outliers=False)
    q = queries(torch, (1, 4, 50, 64), 5) * 0.25
    ws = tq.chunk_workspace(1, 4, 2, 64, 50, 400)
    got = tq.tq_sdpa_chunk(c, q, torch.tensor([400], dtype=torch.int32, device="cuda"), 400, scale, ws)
    check(torch, got, reference(torch, c, q, [400], [50], scale), [50])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_rows_hold_anything(D):
    """Scales and biases that are no numbers in rows that a query row does not attend to leave it as it was."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens, n = [500, 300], 200
    c = make_cache(tq, torch, 2, 2, D, 500, seed=4, capacity=512)
    q = queries(torch, (2, 8, n, D), 6)
    clean = attend(torch, tq, c, q, lens)
    windowed = attend(torch, tq, c, q, lens, window=100)
    for a in (c.k_scale, c.v_scale, c.k_bias, c.v_bias):
        a[0, :, 450] = math.inf     # seen by the last rows only
        a[0, :, 500:] = math.nan
        a[1, :, 300:] = math.nan
        a[1, 0, 0] = -math.inf      # before every window
    for t, want in ((attend(torch, tq, c, q, lens), clean), (attend(torch, tq, c, q, lens, window=100), windowed)):
        assert torch.equal(t[0, :150], want[0, :150])  # positions 300 to 449
        assert torch.equal(t[1, :, 4:], want[1, :, 4:])
    assert torch.equal(attend(torch, tq, c, q, lens, window=100)[1, :, :4], windowed[1, :, :4])


def test_values_at_the_end_of_fp16():
    """Rows whose scale * code + bias passes 65,504 by its rounding."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 1, 64, 16, seed=4)
    for a, x in ((c.v_scale, 8736.0), (c.v_bias, -65504.0), (c.k_scale, 0.0), (c.k_bias, 1.0)):
        a.fill_(x)
    c.v_codes.fill_(0xFF)
    q = queries(torch, (1, 2, 3, 64), 6)
    got = attend(torch, tq, c, q, [16])
    assert bool((got == 65504.0).all())  # 8736 * 15 - 65504 = 65,536


def test_against_single_tokens():
    """Row i of a chunk is the decode of its token over the rows before it."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    n, L, D = 6, 800, 128
    c = make_cache(tq, torch, 2, 2, D, L, seed=9)
    q = queries(torch, (2, 16, n, D), 8)
    got = attend(torch, tq, c, q, [L, 500])
    ws = tq.workspace(2, 16, 2, D, L)
    for i in range(n):
        lens = torch.tensor([L - n + 1 + i, 500 - n + 1 + i], dtype=torch.int32, device="cuda")
        one = tq.tq_sdpa_int4_decode(c, q[:, :, i].contiguous(), lens, L, 1 / math.sqrt(D), ws)
        # the decode rounds no key: what a chunk's rounding may add (see check) and the decode's own 1e-3
        want = reference(torch, c, q[:, :, i:i + 1], lens.tolist(), [1, 1], 1 / math.sqrt(D))
        own = 2 * math.sqrt(float(want[2].sum()))
        assert float((got[:, i].double() - one.double()).norm()) <= own + 1e-3 * float(one.double().norm())


@pytest.mark.parametrize("B,Hq,Hkv,D,bits,n,L,paged", [(1, 64, 8, 128, 4, 8, 131072, False), (1, 64, 8, 128, 4, 3, 131072, True),
                                                       (3, 16, 4, 128, 4, 1024, 5000, True), (1, 8, 1, 64, 8, 1000, 40000, False),
                                                       (2, 12, 6, 256, 4, 700, 3001, False), (12, 64, 8, 128, 8, 100, 2000, True),
                                                       (1, 4, 4, 256, 8, 40, 60000, False), (40, 16, 8, 64, 4, 40, 900, True)])
def test_larger(B, Hq, Hkv, D, bits, n, L, paged):
    """Sequences cut over many CTAs, batches of several waves."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, B, Hkv, D, L, bits, paged, seed=L)
    lens = [max(n, L - 97 * b) for b in range(B)]
    q = queries(torch, (B, Hq, n, D), n)
    check(torch, attend(torch, tq, c, q, lens), reference(torch, c, q, lens, [n] * B, 1 / math.sqrt(D)), [n] * B)


def test_length_reports():
    """Lengths outside their bounds are clamped and reported."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 3, 2, 64, 200, seed=3, capacity=208)
    q = queries(torch, (3, 2, 10, 64), 1)
    want = attend(torch, tq, c, q, [200, 0, 120], [10, 10, 0], max_len=200)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attend(torch, tq, c, q, [999, -5, 120], [99, 10, -1], max_len=200, status=st, out=torch.zeros_like(want))
    assert torch.equal(got[:2], want[:2]) and int(st) == tq.TQ_DEV_SEQ_LEN


def test_bad_pages():
    """A table entry outside the pool reads page 0 and is reported."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 2, 128, 500, paged=True, seed=3)
    q = queries(torch, (1, 4, 30, 128), 1)
    table = c.block_table.clone()
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        c.block_table.copy_(table)
        c.block_table[0, 1] = 0
        want = attend(torch, tq, c, q, [500])
        c.block_table[0, 1] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(attend(torch, tq, c, q, [500], status=st), want) and int(st) == tq.TQ_DEV_PAGE


@pytest.mark.parametrize("n,L", [(4, 9000), (300, 1000)])
def test_graphs_and_streams(n, L):
    """Captured, replayed over new lengths and queries, and on another stream."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 2, 2, 128, L, seed=5)
    q = queries(torch, (2, 8, n, 128), 1)
    lens = torch.tensor([L, L // 2], dtype=torch.int32, device="cuda")
    ws, out = tq.chunk_workspace(2, 8, 2, 128, n, L), torch.zeros((2, n, 8, 128), dtype=torch.float16, device="cuda")
    call = lambda **kw: tq.tq_sdpa_chunk(c, q, lens, L, 0.1, ws, **kw)  # noqa: E731
    call(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out)
    for seed in range(3):
        q.copy_(queries(torch, q.shape, seed + 20))
        lens.copy_(torch.tensor([L - seed, n + seed], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=other)
    other.synchronize()
    assert torch.equal(got, out)


def test_large_offsets():
    """Rows behind 2^32 bytes of a cache."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    cap, D = 1 << 24, 256
    c = tq.KVCache(3, 1, D, cap)
    small = make_cache(tq, torch, 1, 1, D, 400, seed=6)
    at = cap - 400
    for name in ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias"):
        getattr(c, name)[2, :, at:cap] = getattr(small, name)[0, :, :400]
    q = queries(torch, (3, 2, 50, D), 1)
    ws = tq.chunk_workspace(3, 2, 1, D, 50, cap)
    lens = torch.tensor([0, 0, cap], dtype=torch.int32, device="cuda")
    got = tq.tq_sdpa_chunk(c, q, lens, cap, 0.05, ws, window=351)[2]  # the last 400 rows and no others
    want = reference(torch, small, q[2:], [400], [50], 0.05, 351)
    check(torch, got.unsqueeze(0), want, [50])


def test_nothing_to_do():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 2, 64, 16, seed=6)
    ws = tq.chunk_workspace(1, 4, 2, 64, 1, 16)
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    assert tq.tq_sdpa_chunk(c, queries(torch, (1, 4, 0, 64), 1), lens, 16, 1.0, ws).shape == (1, 0, 4, 64)
