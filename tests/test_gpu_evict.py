"""Eviction by accumulated weight, compared exactly (rows are copied, indices
are whole numbers), and the operators of a decode loop one after another."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import assert_close, need_gpu
from tests.operator_helpers import dev, host, make_cache, rows, softmax_rows, values

pytestmark = pytest.mark.gpu

ARRAYS = ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias")
LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]


def kept_reference(w, n, keep, recent):
    """Rows that stay of one head's weights [n]."""
    if n <= keep:
        return np.arange(n)
    old = n - recent
    best = np.argsort(-(w[:old].astype(np.float64) + 0.0), kind="stable")[: keep - recent]
    return np.concatenate([np.sort(best), np.arange(old, n)])


def evict_and_check(tq, torch, src, dst, w, lens, max_len, keep, recent):
    B, Hkv = src.batch, src.num_kv_heads
    dw = torch.full((B, Hkv, dst.capacity), 9.0, device="cuda")
    dl = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((B, Hkv, keep), -9, dtype=torch.int32, device="cuda")
    before = {a: rows(dst, a).copy() for a in ARRAYS}
    source = {a: rows(src, a).copy() for a in ARRAYS}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(src, dst, dev(torch, w), dev(torch, np.asarray(lens, np.int32)), max_len, keep, recent, dw, dl, kept, status=st)
    kept, dw, dl = kept.cpu().numpy(), dw.cpu().numpy(), dl.cpu().numpy()
    after = {a: rows(dst, a) for a in ARRAYS}
    for b in range(B):
        n = min(max(int(lens[b]), 0), max_len)
        assert dl[b] == min(n, keep)
        for h in range(Hkv):
            want = kept_reference(w[b, h], n, keep, recent)
            m = len(want)
            assert np.array_equal(kept[b, h, :m], want), (b, h)
            assert (kept[b, h, m:] == -1).all()
            assert np.array_equal(dw[b, h, :m], w[b, h, want]) and not dw[b, h, m:].any()
            for a in ARRAYS:
                assert np.array_equal(after[a][b, h, :m].view(np.uint8), source[a][b, h, want].view(np.uint8)), a
                assert np.array_equal(after[a][b, h, m:].view(np.uint8), before[a][b, h, m:].view(np.uint8)), a
    return int(st)


def heavy(rng, shape):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    w[rng.random(shape) < 0.1] = 0.0
    return w


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (100, 17), (257, 0), (300, 300), (600, 64), (1000, 10)])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_evict(D, bits, keep, recent, paged):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n = 4, 2, 900
    src = make_cache(tq, torch, B, Hkv, D, n, bits, paged, seed=D + keep, capacity=1024)
    dst = make_cache(tq, torch, B, Hkv, D, 16, bits, paged, seed=1, capacity=1024)
    rng = np.random.default_rng(keep)
    w = heavy(rng, (B, Hkv, src.capacity))
    assert evict_and_check(tq, torch, src, dst, w, [n, 0, 1, 611], n, keep, recent) == 0


@pytest.mark.parametrize("n,keep,recent", [(131072, 4096, 256), (50000, 1000, 0), (4097, 4096, 1), (9001, 33, 32), (400000, 3000, 100)])
def test_evict_long(n, keep, recent):
    """Several CTAs a head; 400,000 weights do not fit their registers."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    Hkv = 1 if n > 200000 else 2
    src, dst = tq.KVCache(1, Hkv, 64, -(-n // 16) * 16), tq.KVCache(1, Hkv, 64, 4096)
    src.buffer.random_(0, 256)
    dst.buffer.zero_()
    rng = np.random.default_rng(n)
    evict_and_check(tq, torch, src, dst, heavy(rng, (1, Hkv, src.capacity)), [n], n, keep, recent)


@pytest.mark.parametrize("n,keep,recent", [(131072, 4096, 256), (150001, 70000, 5)])
@pytest.mark.parametrize("kind", ["equal", "two values", "narrow"])
def test_evict_long_ties(kind, n, keep, recent):
    """More keys of one digit than the CTAs of a head send each other, down to the last bit."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    src, dst = tq.KVCache(1, 2, 64, -(-n // 16) * 16), tq.KVCache(1, 2, 64, -(-keep // 16) * 16)
    src.buffer.random_(0, 256)
    dst.buffer.zero_()
    rng = np.random.default_rng(n)
    shape = (1, 2, src.capacity)
    w = {"equal": np.full(shape, 3.5), "two values": rng.integers(0, 2, shape) * 0.5,
         "narrow": 1.0 + rng.integers(0, 30, shape) * 2.0 ** -23}[kind].astype(np.float32)
    evict_and_check(tq, torch, src, dst, w, [n], n, keep, recent)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("keep,recent", [(640, 640), (640, 500)])
def test_evict_between_appends(keep, recent, graph):
    """Rows that the weights do not decide are copied beside the selection, but after the append before the call and before the
    one behind it: nothing is waited for on the host."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, D, n, cap = 3, 2, 128, 2000, 2048
    src, dst = make_cache(tq, torch, B, Hkv, D, 0, seed=8, capacity=cap), make_cache(tq, torch, B, Hkv, D, 0, seed=9, capacity=1024)
    rng = np.random.default_rng(keep + recent)
    rows_of = [dev(torch, rng.standard_normal((2, B, Hkv, n, D)).astype(np.float16)) for _ in range(4)]
    zero, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), dev(torch, np.array([n, 1500, 600], np.int32))
    w = dev(torch, heavy(rng, (B, Hkv, cap)))
    dw, dl = torch.zeros((B, Hkv, 1024), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, Hkv, keep), dtype=torch.int32, device="cuda")
    want = []
    for x in rows_of:
        tq.tq_quantize_kv_append(src, x[0], x[1], zero)
        want.append(rows(src, "v_codes"))
    got = [torch.empty_like(dst.v_codes) for _ in rows_of]

    def go():
        for x, g in zip(rows_of, got):
            tq.tq_quantize_kv_append(src, x[0], x[1], zero)
            tq.tq_kv_evict(src, dst, w, lens, n, keep, recent, dw, dl, kept)
            tq.tq_quantize_kv_append(src, rows_of[0][1], rows_of[0][0], zero)
            g.copy_(dst.v_codes)

    if graph:
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            go()
        c.replay()
    else:
        go()
    for x, g in zip(want, got):
        for b, ln in enumerate((n, 1500, 600)):
            for h in range(Hkv):
                r = kept_reference(w.cpu().numpy()[b, h], ln, keep, recent)
                assert np.array_equal(g.cpu().numpy()[b, h, : len(r)], x[b, h, r])


@pytest.mark.parametrize("kind", ["equal", "two values", "signed zeros", "negative", "infinite", "tiny steps"])
def test_evict_ties_and_odd_weights(kind):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n, keep, recent = 2, 3, 9000, 700, 50
    src, dst = make_cache(tq, torch, B, Hkv, 64, n, seed=3), make_cache(tq, torch, B, Hkv, 64, 16, capacity=1024)
    rng = np.random.default_rng(11)
    shape = (B, Hkv, src.capacity)
    w = {"equal": np.full(shape, 0.25), "two values": rng.integers(0, 2, shape) * 0.5, "signed zeros": np.where(rng.random(shape) < 0.5, 0.0, -0.0),
         "negative": -rng.random(shape), "infinite": np.where(rng.random(shape) < 0.1, np.inf, rng.random(shape)),
         "tiny steps": 1.0 + rng.integers(0, 3000, shape) * 2.0 ** -23}[kind].astype(np.float32)
    evict_and_check(tq, torch, src, dst, w, [n, n - 1], n, keep, recent)


def test_evict_weights_that_are_no_numbers_end_in_bounds():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    src, dst = make_cache(tq, torch, 1, 2, 64, 5000, seed=3), make_cache(tq, torch, 1, 2, 64, 16, capacity=512)
    w = np.random.default_rng(1).random((1, 2, src.capacity)).astype(np.float32)
    w[:, :, ::5] = np.nan
    w[:, :, 1::5] = -np.nan
    dw, dl = torch.zeros((1, 2, 512), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros((1, 2, 300), dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(src, dst, dev(torch, w), dev(torch, np.array([5000], np.int32)), 5000, 300, 20, dw, dl, kept)
    k = kept.cpu().numpy()
    assert ((k >= 0) & (k < 5000)).all() and (np.diff(k, axis=-1) > 0).all()


def test_evict_lengths_outside_are_clamped_and_reported():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    src, dst = make_cache(tq, torch, 3, 2, 128, 300, seed=4), make_cache(tq, torch, 3, 2, 128, 16, capacity=128)
    w = heavy(np.random.default_rng(4), (3, 2, src.capacity))
    assert evict_and_check(tq, torch, src, dst, w, [301, -1, 250], 250, 100, 10) == tq.TQ_DEV_SEQ_LEN


def test_evict_in_a_graph():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n, keep = 2, 2, 6000, 500
    src, dst = make_cache(tq, torch, B, Hkv, 128, n, seed=5), make_cache(tq, torch, B, Hkv, 128, 16, capacity=512)
    rng = np.random.default_rng(5)
    w, lens = dev(torch, heavy(rng, (B, Hkv, src.capacity))), dev(torch, np.array([n, 4000], np.int32))
    dw, dl = torch.zeros((B, Hkv, 512), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, Hkv, keep), dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(src, dst, w, lens, n, keep, 40, dw, dl, kept)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_kv_evict(src, dst, w, lens, n, keep, 40, dw, dl, kept)
    w2 = heavy(rng, (B, Hkv, src.capacity))
    w.copy_(dev(torch, w2))
    lens.copy_(dev(torch, np.array([300, 5999], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    got = kept.cpu().numpy()
    for b, ln in enumerate((300, 5999)):
        for h in range(Hkv):
            want = kept_reference(w2[b, h], ln, keep, 40)
            assert np.array_equal(got[b, h, : len(want)], want)
            assert np.array_equal(rows(dst, "k_codes")[b, h, : len(want)], rows(src, "k_codes")[b, h, want])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
def test_a_decode_loop(bits, paged):
    """A prompt and some tokens as a serving loop would take them: rotary positions, append, bounds, a sparse step and a full step
    that keeps the weights; then eviction, and another step over what is left.  Each output against fp64 over the cache as it
    stands."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, prompt, steps, block, K = 2, 16, 2, 128, 700, 5, 64, 6
    scale, cap = 1 / math.sqrt(D), 1024
    rng = np.random.default_rng(bits)
    c = make_cache(tq, torch, B, Hkv, D, 0, bits, paged, seed=6, capacity=cap)
    bounds, w = tq.block_bounds(c, block), torch.zeros((B, Hkv, cap), device="cuda")
    inv = dev(torch, (500000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
    ws = tq.sparse_workspace(B, Hq, Hkv, D, cap, K, block)
    wws = tq.weights_workspace(B, Hq, Hkv, D, cap)
    blocks = torch.zeros((B, Hkv, K), dtype=torch.int32, device="cuda")
    pos_at = np.zeros(B, np.int32)

    def take(n):
        """n new tokens of every sequence: their query heads [B, Hq, n, D], appended."""
        qkv = dev(torch, rng.standard_normal((B, n, Hq + 2 * Hkv, D)).astype(np.float16))
        t = pos_at[:, None] + np.arange(n)
        pos = dev(torch, np.stack([t, t // 8, t % 8]).astype(np.int32))
        q, k = tq.tq_rope_axes(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], pos, inv, (16, 24, 24))
        v = qkv[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
        at = dev(torch, pos_at)
        tq.tq_quantize_kv_append(c, k, v, at)
        tq.tq_kv_block_bounds(c, bounds, at, n, block_tokens=block)
        pos_at[:] += n
        return q

    take(prompt)
    total = np.zeros((B, Hkv, cap))
    for _ in range(steps):
        q = take(1)[:, :, 0].contiguous()
        lens = dev(torch, pos_at)
        sparse, _ = tq.tq_sparse_decode(c, bounds, q, lens, cap, scale, ws, blocks, block_tokens=block)
        dense = tq.tq_sdpa_decode_weights(c, q, lens, cap, scale, w, wws)
        k, v, qh, bl = values(c, "k"), values(c, "v"), host(q), blocks.cpu().numpy()
        n = int(pos_at[0])
        for b in range(B):
            for h in range(Hkv):
                g = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
                o, p = softmax_rows(qh[b, g], k[b, h, :n], v[b, h, :n], scale)
                assert_close(host(dense)[b, g], o)
                total[b, h, :n] += p.sum(0)
                lo, hi = (np.stack([getattr(k[b, h, j:min(j + block, n)].astype(np.float16), m)(0) for j in range(0, n, block)]) for m in ("min", "max"))
                s = np.maximum(qh[b, g, None] * lo, qh[b, g, None] * hi).sum(-1).max(0)
                mid = np.argsort(-s[1:-1], kind="stable")[: K - 2] + 1
                want = np.concatenate([[0], np.sort(mid), [len(s) - 1]])
                assert np.array_equal(bl[b, h], want)
                r = (want[:, None] * block + np.arange(block)).ravel()
                r = r[r < n]
                assert_close(host(sparse)[b, g], softmax_rows(qh[b, g], k[b, h, r], v[b, h, r], scale)[0])
    got = w.cpu().numpy()
    n = int(pos_at[0])
    assert np.linalg.norm(got[:, :, :n] - total[:, :, :n]) <= 1e-5 * np.linalg.norm(total)
    keep, recent = 200, 40
    small = make_cache(tq, torch, B, Hkv, D, 0, bits, paged, seed=7, capacity=256)
    sw, sl = torch.zeros((B, Hkv, small.capacity), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, Hkv, keep), dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(c, small, w, dev(torch, pos_at), cap, keep, recent, sw, sl, kept)
    q = dev(torch, rng.standard_normal((B, Hq, D)).astype(np.float16))
    kn = dev(torch, rng.standard_normal((B, Hkv, 1, D)).astype(np.float16))
    at = sl.clone()
    out = tq.tq_decode_step(small, kn, kn, at, q, sl + 1, small.capacity, scale, tq.workspace(B, Hq, Hkv, D, small.capacity))
    k, v, qh = values(small, "k"), values(small, "v"), host(q)
    for b in range(B):
        for h in range(Hkv):
            want = kept_reference(got[b, h], n, keep, recent)
            assert np.array_equal(kept.cpu().numpy()[b, h], want)
            assert np.array_equal(rows(small, "k_codes")[b, h, :keep], rows(c, "k_codes")[b, h, want])
            g = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
            assert_close(host(out)[b, g], softmax_rows(qh[b, g], k[b, h, : keep + 1], v[b, h, : keep + 1], scale)[0])
