"""Block bounds, block selection and decode attention over listed blocks
against fp64 (tests/operator_helpers.py).

Bounds are compared exactly: scale * code + bias is exact in fp64 and rounded
once to fp16 on both sides.  Selections are compared exactly: the reference
orders fp64 scores (fp16 products are exact there; the scores of the inputs
here differ by far more than the 2^-45 their sums are off, or are equal).
Attention outputs are held to the decode's own bounds (ATOL, RTOL_L2 of
tests/gpu_helpers.py): the kernel's arithmetic on a row is the decode's."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import assert_close, need_gpu
from tests.operator_helpers import dev, host, make_cache, softmax_rows, values

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]


# ---------------------------------------------------------------------- bounds
def bounds_reference(cache, block, start, n_rows, before):
    k = values(cache, "k")
    out = before.copy()
    for b in range(cache.batch):
        stop = int(start[b]) + n_rows
        for j in range(int(start[b]) // block, -(-stop // block)):
            part = k[b, :, j * block: min((j + 1) * block, stop)].astype(np.float16)
            out[b, :, j, 0], out[b, :, j, 1] = part.min(1), part.max(1)
    return out


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_bounds_of_a_prompt_and_of_steps(D, bits, block, paged):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n = 2, 3, 397
    c = make_cache(tq, torch, B, Hkv, D, n, bits, paged, seed=D + block, capacity=400)
    bounds = tq.block_bounds(c, block)
    bounds.fill_(7.0)
    before = bounds.cpu().numpy()
    for start, rows in (([0, 0], n), ([5, 131], 1), ([31, 63], 200), ([396, 0], 1)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        tq.tq_kv_block_bounds(c, bounds, dev(torch, np.array(start, np.int32)), rows, block_tokens=block, status=st)
        want = bounds_reference(c, block, start, rows, before)
        got = bounds.cpu().numpy()
        assert np.array_equal(got, want)  # touched blocks recomputed, the others as they were
        assert int(st) == 0
        before = got


def test_bounds_ranges_outside_the_cache():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 3, 2, 128, 64, seed=1, capacity=80)
    bounds = tq.block_bounds(c, 32)
    bounds.fill_(3.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = np.array([-1, 79, 10], np.int32)
    tq.tq_kv_block_bounds(c, bounds, dev(torch, start), 2, block_tokens=32, status=st)
    got = bounds.cpu().numpy()
    assert int(st) == tq.TQ_DEV_WRITE_POS
    assert (got[:2] == 3.0).all()
    want = bounds_reference(c, 32, [0, 0, 10], 2, np.full_like(got, 3.0))
    assert np.array_equal(got[2], want[2])
    tq.tq_kv_block_bounds(c, bounds, dev(torch, start), 0, block_tokens=32)  # nothing


# ------------------------------------------------------------------- selection
def scores_reference(bounds, q):
    """fp64 [B, Hkv, nb]."""
    B, Hkv = bounds.shape[:2]
    g = q.reshape(B, Hkv, -1, 1, q.shape[-1]).astype(np.float64)
    lo, hi = bounds[:, :, None, :, 0].astype(np.float64), bounds[:, :, None, :, 1].astype(np.float64)
    return np.maximum(g * lo, g * hi).sum(-1).max(2)


def select_reference(scores, lens, block, K, first, last):
    B, H = scores.shape[:2]
    out = np.full((B, H, K), -1, np.int32)
    for b in range(B):
        nb = -(-int(lens[b]) // block)
        for h in range(H):
            if nb <= K:
                pick = np.arange(nb)
            else:
                mid = np.argsort(-scores[b, h, first: nb - last], kind="stable")[: K - first - last] + first
                pick = np.sort(np.concatenate([np.arange(first), mid, np.arange(nb - last, nb)]))
            out[b, h, : len(pick)] = pick
    return out


def run_select(tq, torch, bounds, q, lens, max_len, block, K, first, last, capacity, status=None):
    B, Hkv = bounds.shape[:2]
    ws = tq.sparse_workspace(B, q.shape[1], Hkv, q.shape[2], max_len, K, block)
    blocks = torch.full((B, Hkv, K), -7, dtype=torch.int32, device="cuda")
    tq.tq_select_blocks(dev(torch, bounds), dev(torch, q), dev(torch, np.asarray(lens, np.int32)), max_len, ws, blocks, capacity,
                        block_tokens=block, n_first=first, n_last=last, status=status)
    return blocks.cpu().numpy()


def random_bounds(rng, B, H, nb, D):
    x = rng.standard_normal((2, B, H, nb, D)) * 2
    return np.stack((x.min(0), x.max(0)), 3).astype(np.float16)


@pytest.mark.parametrize("D,G,Hkv,B,block,cap,K,first,last", [
    (128, 8, 8, 1, 64, 131072, 64, 1, 1), (128, 8, 4, 3, 32, 4096, 16, 1, 1), (64, 1, 2, 4, 128, 20000, 9, 2, 3),
    (256, 2, 3, 2, 32, 3008, 5, 0, 0), (128, 3, 1, 5, 64, 9600, 7, 0, 1), (64, 7, 2, 2, 32, 65536, 100, 4, 60),
    (128, 5, 2, 2, 64, 1040, 1, 0, 0), (128, 8, 2, 2, 64, 1040, 3, 3, 0), (64, 4, 1, 1, 32, 32 * 5000, 64, 1, 1),
])
def test_selection_matches_the_exact_order(D, G, Hkv, B, block, cap, K, first, last):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(cap + D)
    nb = -(-cap // block)
    bounds = random_bounds(rng, B, Hkv, nb, D)
    q = rng.standard_normal((B, Hkv * G, D)).astype(np.float16)
    lens = np.array([cap, 0, 1, cap // 3, K * block + 1][:B] if B > 1 else [cap], np.int32)
    got = run_select(tq, torch, bounds, q, lens, cap, block, K, first, last, cap)
    assert np.array_equal(got, select_reference(scores_reference(bounds, q), lens, block, K, first, last))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_selection_near_and_equal_scores(D):
    """Blocks that repeat (equal scores: the lowest index first), and blocks one fp16 step of one small channel apart, whose fp32
    sums are not to be told apart: the order is the exact one."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(D)
    B, H, G, block, nb = 2, 2, 4, 64, 700
    one = random_bounds(rng, B, H, 1, D)
    one[..., 0] = np.float16(-60.0), np.float16(55.0)  # not used below
    bounds = np.repeat(one, nb, 2)
    bounds[:, :, :, 0, 0], bounds[:, :, :, 1, 0] = -60.0, 55.0  # an outlier channel sets the sums' size
    # channel 1: steps of 2^-14 around zero, most of them repeated
    bounds[:, :, :, 1, 1] = (rng.integers(0, 40, (B, H, nb)) * 2.0 ** -14).astype(np.float16)
    bounds[:, :, :, 0, 1] = 0
    q = rng.standard_normal((B, H * G, D)).astype(np.float16)
    q[:, :, 1] = np.float16(2.0 ** -7) * rng.integers(1, 4, (B, H * G))
    lens = np.array([nb * block, nb * block - 70], np.int32)
    for K in (2, 37, 333):
        got = run_select(tq, torch, bounds, q, lens, nb * block, block, K, 1, 1, nb * block)
        assert np.array_equal(got, select_reference(scores_reference(bounds, q), lens, block, K, 1, 1)), K


@pytest.mark.parametrize("scale_q,scale_b", [(1.0, 2.0 ** -20), (2.0 ** -20, 1.0), (2.0 ** -18, 2.0 ** -18), (1e-3, 2.0 ** -16)])
def test_selection_of_subnormal_numbers(scale_q, scale_b):
    """fp16 subnormals, whose products the tensor core sums with fewer bits: still the exact order."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(77)
    B, H, G, D, block, nb, K = 2, 2, 4, 128, 32, 1500, 40
    x = rng.standard_normal((2, B, H, nb, D)) * 8 * scale_b
    bounds = np.stack((x.min(0), x.max(0)), 3).astype(np.float16)
    q = (rng.standard_normal((B, H * G, D)) * 4 * scale_q).astype(np.float16)
    got = run_select(tq, torch, bounds, q, [nb * block, nb * block - 5], nb * block, block, K, 1, 1, nb * block)
    assert np.array_equal(got, select_reference(scores_reference(bounds, q), [nb * block, nb * block - 5], block, K, 1, 1))


def test_selection_ignores_the_bounds_of_listed_blocks_and_clamps_lengths():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(9)
    bounds = random_bounds(rng, 3, 2, 64, 128)
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    want = select_reference(scores_reference(bounds, q), [4096, 4096, 0], 64, 12, 2, 2)
    for bad in (np.nan, np.inf, -np.inf):
        b2 = bounds.copy()
        b2[:, :, :2] = bad
        b2[:, :, -2:] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_select(tq, torch, b2, q, [4096, 5000, -3], 4096, 64, 12, 2, 2, 4096, status=st)
        assert np.array_equal(got, want)
        assert int(st) == tq.TQ_DEV_SEQ_LEN


def test_selection_of_scores_that_are_no_numbers_ends_in_bounds():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(10)
    bounds = random_bounds(rng, 1, 2, 300, 64)
    bounds[:, :, ::3] = np.nan
    bounds[:, :, 1::7] = np.inf
    q = rng.standard_normal((1, 4, 64)).astype(np.float16)
    got = run_select(tq, torch, bounds, q, [300 * 64], 300 * 64, 64, 20, 1, 1, 300 * 64)
    assert ((got >= -1) & (got < 300)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_selection_with_infinite_bounds(D):
    """Keys above fp16's range (an infinite greatest or least key): a head that turns away from the channel scores by the other
    bound, a channel of zero adds nothing, and infinite scores come first, the lowest index first."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    rng = np.random.default_rng(D + 7)
    B, H, G, block, nb, K = 2, 2, 3, 64, 333, 20
    bounds = random_bounds(rng, B, H, nb, D)
    bounds[:, :, 5::9, 1, 3] = np.inf
    bounds[0, :, 7::31, 0, 4] = -np.inf
    q = rng.standard_normal((B, H * G, D)).astype(np.float16)
    q[:, :, 3] = -np.abs(q[:, :, 3]) - np.float16(0.25)  # nobody gains from the infinite channel 3 ...
    q[1, 1, 3] = 1.0                                     # ... but one head
    q[0, :, 4] = 0.0                                     # channel 4 counts for nobody
    g, lo, hi = (x.astype(np.float64) for x in (q.reshape(B, H, G, 1, D), bounds[:, :, None, :, 0], bounds[:, :, None, :, 1]))
    with np.errstate(invalid="ignore"):
        scores = np.where(g == 0, 0.0, np.where(g > 0, g * hi, g * lo)).sum(-1).max(2)
    assert np.isinf(scores[1, 0]).any() and np.isfinite(scores[0]).all() and not np.isnan(scores).any()
    got = run_select(tq, torch, bounds, q, [nb * block] * B, nb * block, block, K, 1, 1, nb * block)
    assert np.array_equal(got, select_reference(scores, [nb * block] * B, block, K, 1, 1))


# ------------------------------------------------------------ listed attention
def attend_reference(cache, q, blocks, lens, block, scale, flags=0, tq=None):
    k, v = values(cache, "k"), values(cache, "v")
    B, Hkv, D = cache.batch, cache.num_kv_heads, cache.head_dim
    G = q.shape[1] // Hkv
    out = np.zeros(q.shape)
    for b in range(B):
        for h in range(Hkv):
            r = [np.arange(j * block, min((j + 1) * block, int(lens[b]))) for j in blocks[b, h].tolist() if 0 <= j and j * block < lens[b]]
            r = np.concatenate(r) if r else np.zeros(0, int)
            out[b, h * G:(h + 1) * G] = softmax_rows(q[b, h * G:(h + 1) * G].astype(np.float64), k[b, h, r], v[b, h, r], scale)[0]
    return out


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_listed_blocks(D, bits, block, paged):
    """Lists in any order, with empty entries, repeats, partial and missing blocks."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, G, n = 4, 2, 5, 1000
    c = make_cache(tq, torch, B, Hkv, D, n, bits, paged, seed=D + block + bits)
    rng = np.random.default_rng(block)
    nb = -(-n // block)
    q = rng.standard_normal((B, Hkv * G, D)).astype(np.float16)
    lens = np.array([n, 0, 1, n - 37], np.int32)
    K = 11
    blocks = rng.integers(-1, nb, (B, Hkv, K)).astype(np.int32)
    blocks[0, 0] = -1                     # an empty list
    blocks[0, 1] = np.arange(K) % nb
    blocks[3, 0, 5:] = (nb - 1, nb - 1, 0, -1, 2 ** 31 - 1, -2 ** 31)  # the partial block twice, one past the end
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = tq.sparse_workspace(B, Hkv * G, Hkv, D, n, K, block)
    out = tq.tq_sdpa_blocks_decode(c, dev(torch, q), dev(torch, blocks), dev(torch, lens), n, 1 / math.sqrt(D), ws,
                                   block_tokens=block, status=st)
    want = attend_reference(c, q, blocks, lens, block, 1 / math.sqrt(D))
    got = host(out)
    assert_close(got, want, what=f"D={D} bits={bits} block={block}")
    assert not got[0, :G].any() and not got[1].any()
    assert int(st) == tq.TQ_DEV_BLOCK


@pytest.mark.parametrize("B,Hq,Hkv,D,K", [(1, 64, 8, 128, 64), (1, 1, 1, 128, 1), (2, 8, 1, 64, 300), (32, 64, 16, 64, 2100),
                                          (1, 32, 16, 256, 7), (7, 24, 8, 128, 33)])
def test_every_plan(B, Hq, Hkv, D, K):
    """One run, runs merged by a cluster, partial states and the reduce; lists longer than a run's window (repeats count)."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    n, block = 640, 32
    c = make_cache(tq, torch, B, Hkv, D, n, 4, False, seed=K)
    rng = np.random.default_rng(K)
    q = rng.standard_normal((B, Hq, D)).astype(np.float16)
    lens = rng.integers(n // 2, n + 1, B).astype(np.int32)
    blocks = rng.integers(0, n // block // 2, (B, Hkv, K)).astype(np.int32)
    ws = tq.sparse_workspace(B, Hq, Hkv, D, n, K, block)
    out = tq.tq_sdpa_blocks_decode(c, dev(torch, q), dev(torch, blocks), dev(torch, lens), n, 1 / math.sqrt(D), ws, block_tokens=block)
    # a block listed c times counts c times: weights by log(c) on its scores, the same sum
    k, v = values(c, "k"), values(c, "v")
    G = Hq // Hkv
    want = np.zeros((B, Hq, D))
    for b in range(B):
        for h in range(Hkv):
            count = np.repeat(np.bincount(blocks[b, h], minlength=n // block), block)[: lens[b]]
            s = (q[b, h * G:(h + 1) * G].astype(np.float64) @ k[b, h, : lens[b]].T) / math.sqrt(D)
            p = np.exp(s - s.max()) * count
            want[b, h * G:(h + 1) * G] = (p / p.sum(-1, keepdims=True)) @ v[b, h, : lens[b]]
    assert_close(host(out), want)


@pytest.mark.parametrize("paged", [False, True])
def test_all_blocks_are_the_decode(paged):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, n = 2, 16, 2, 128, 1500
    c = make_cache(tq, torch, B, Hkv, D, n, 4, paged, seed=2)
    rng = np.random.default_rng(2)
    q, lens = dev(torch, rng.standard_normal((B, Hq, D)).astype(np.float16)), dev(torch, np.array([n, 700], np.int32))
    bounds = tq.block_bounds(c, 64)
    tq.tq_kv_block_bounds(c, bounds, torch.zeros(B, dtype=torch.int32, device="cuda"), n)
    blocks = torch.zeros((B, Hkv, 30), dtype=torch.int32, device="cuda")
    ws = tq.sparse_workspace(B, Hq, Hkv, D, n, 30)
    out, _ = tq.tq_sparse_decode(c, bounds, q, lens, n, 0.1, ws, blocks)
    dense = tq.tq_sdpa_int4_decode(c, q, lens, n, 0.1, tq.workspace(B, Hq, Hkv, D, n))
    assert_close(host(out), host(dense))
    assert np.array_equal(blocks.cpu().numpy()[1, 0], np.concatenate([np.arange(11), np.full(19, -1)]))


@pytest.mark.parametrize("flags", [1, 2, 3])
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_sparse_decode_of_a_rotated_cache(D, bits, flags):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, n, block, K = 2, 12, 2, 1111, 32, 9
    c = make_cache(tq, torch, B, Hkv, D, n, bits, seed=D + flags, flags=flags)
    rng = np.random.default_rng(D)
    q = rng.standard_normal((B, Hq, D)).astype(np.float16)
    lens = np.array([n, 555], np.int32)
    bounds = tq.block_bounds(c, block)
    tq.tq_kv_block_bounds(c, bounds, torch.zeros(B, dtype=torch.int32, device="cuda"), n, block_tokens=block)
    blocks = torch.zeros((B, Hkv, K), dtype=torch.int32, device="cuda")
    ws = tq.sparse_workspace(B, Hq, Hkv, D, n, K, block)
    qt = dev(torch, q)
    out, _ = tq.tq_sparse_decode(c, bounds, qt, dev(torch, lens), n, 1 / math.sqrt(D), ws, blocks, block_tokens=block, flags=flags)
    q_in = host(tq.tq_hadamard_rotate(qt)).astype(np.float16) if flags & tq.TQ_ROTATE_K else q
    b_host = bounds.cpu().numpy()
    b_host[1, :, -(-555 // block):] = 0
    want_blocks = select_reference(scores_reference(b_host, q_in), lens, block, K, 1, 1)
    assert np.array_equal(blocks.cpu().numpy(), want_blocks)
    want = attend_reference(c, q_in, want_blocks, lens, block, 1 / math.sqrt(D))
    if flags & tq.TQ_ROTATE_V:
        H = np.array([[1.0]])
        while H.shape[0] < D:
            H = np.block([[H, H], [H, -H]])
        want = want @ H / math.sqrt(D)
    assert_close(host(out), want)
    alone = tq.tq_sdpa_blocks_decode(c, qt, blocks, dev(torch, lens), n, 1 / math.sqrt(D), ws, block_tokens=block, flags=flags)
    assert_close(host(alone), want)


def test_sparse_decode_in_a_graph_and_on_two_streams():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, n, block, K = 1, 32, 4, 128, 20000, 64, 10
    c = make_cache(tq, torch, B, Hkv, D, n, 4, seed=8)
    rng = np.random.default_rng(8)
    bounds = tq.block_bounds(c, block)
    tq.tq_kv_block_bounds(c, bounds, torch.zeros(B, dtype=torch.int32, device="cuda"), n)
    qs = [rng.standard_normal((B, Hq, D)).astype(np.float16) for _ in range(4)]
    lens = dev(torch, np.array([n], np.int32))
    b_host = bounds.cpu().numpy()

    def expect(q, ln):
        bl = select_reference(scores_reference(b_host, q), [ln], block, K, 1, 1)
        return bl, attend_reference(c, q, bl, [ln], block, 0.09)

    # two calls at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    state = []
    torch.cuda.synchronize()
    for s, q in zip(streams, qs):
        ws, bl = tq.sparse_workspace(B, Hq, Hkv, D, n, K, block), torch.zeros((B, Hkv, K), dtype=torch.int32, device="cuda")
        qt, out = dev(torch, q), torch.zeros((B, Hq, D), dtype=torch.float16, device="cuda")
        torch.cuda.synchronize()
        state.append((ws, bl, qt, out))
    for _ in range(20):
        for s, (ws, bl, qt, out) in zip(streams, state):
            tq.tq_sparse_decode(c, bounds, qt, lens, n, 0.09, ws, bl, out=out, stream=s)
    torch.cuda.synchronize()
    for q, (ws, bl, qt, out) in zip(qs, state):
        wb, wo = expect(q, n)
        assert np.array_equal(bl.cpu().numpy(), wb)
        assert_close(host(out), wo)
    # captured once, replayed with another query and another length
    ws, bl, qt, out = state[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_sparse_decode(c, bounds, qt, lens, n, 0.09, ws, bl, out=out)
    for q, ln in ((qs[2], n), (qs[3], 7777)):
        qt.copy_(dev(torch, q))
        lens.fill_(ln)
        g.replay()
        torch.cuda.synchronize()
        wb, wo = expect(q, ln)
        assert np.array_equal(bl.cpu().numpy(), wb)
        assert_close(host(out), wo)
