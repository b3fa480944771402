"""The decode that accumulates attention weights against fp64.

The output is held to the decode's bounds (tests/gpu_helpers.py).  The weights
are fp32 sums of at most eight probabilities.  A probability's relative error
is that of its score in absolute terms: the score is formed in fp32 from
products whose magnitudes reach S = scale * sum |q_d k_d|, some 30 for these
inputs, each of the NG groups' sums cut at 2^-23 of its magnitude four to eight
times over: at most 8 * 2^-23 * 30 = 3e-5 for a single row, and independent
from row to row.  Over all rows (relative L2) the contract is 1e-5; single
weights are held to 4e-5 of themselves plus 1e-7 of the heads' sum for what
underflows."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import assert_close, need_gpu
from tests.operator_helpers import dev, host, make_cache, softmax_rows, values

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]


def reference(cache, q, lens, scale, old, decay):
    k, v = values(cache, "k"), values(cache, "v")
    G = q.shape[1] // cache.num_kv_heads
    out, w = np.zeros(q.shape), old.astype(np.float64).copy()
    for b in range(cache.batch):
        n = int(lens[b])
        for h in range(cache.num_kv_heads):
            o, p = softmax_rows(q[b, h * G:(h + 1) * G].astype(np.float64), k[b, h, :n], v[b, h, :n], scale)
            out[b, h * G:(h + 1) * G] = o
            w[b, h, :n] = (decay * w[b, h, :n] if decay else 0.0) + p.sum(0)
    return out, w


def check(got, want, lens, G):
    for b, n in enumerate(lens):
        x, y = got[b, :, :n].astype(np.float64), want[b, :, :n]
        assert np.linalg.norm(x - y) <= 1e-5 * np.linalg.norm(y)
        assert (np.abs(x - y) <= 4e-5 * np.abs(y) + 1e-7 * G).all()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("D,bits", LAYOUTS)
def test_weights(D, bits, G, paged):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hkv, n = 4, 2, 900
    c = make_cache(tq, torch, B, Hkv, D, n, bits, paged, seed=D + G, capacity=1024)
    rng = np.random.default_rng(D)
    q = rng.standard_normal((B, Hkv * G, D)).astype(np.float16)
    lens = np.array([n, 0, 1, 517], np.int32)
    old = rng.random((B, Hkv, c.capacity)).astype(np.float32) * 0.01
    ws = tq.weights_workspace(B, Hkv * G, Hkv, D, n)
    for decay in (0.0, 1.0, 0.75):
        w = dev(torch, old)
        if decay == 0.0:
            w.fill_(float("nan"))  # not read
            w[:, :, n:] = 5.0
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = tq.tq_sdpa_decode_weights(c, dev(torch, q), dev(torch, lens), n, 1 / math.sqrt(D), w, ws, decay=decay, status=st)
        want_o, want_w = reference(c, q, lens, 1 / math.sqrt(D), old, decay)
        assert_close(host(out), want_o)
        got = w.cpu().numpy()
        check(got, want_w, lens, G)
        if decay:  # rows at and past the length are left as they were
            for b, ln in enumerate(lens):
                assert np.array_equal(got[b, :, ln:], old[b, :, ln:])
        else:
            assert (got[:, :, n:] == 5.0).all() and np.isnan(got[1, :, 0]).all()
        assert int(st) == 0
        assert not host(out)[1].any()


@pytest.mark.parametrize("B,Hq,Hkv,D,bits,n", [(1, 64, 8, 128, 4, 131072), (8, 64, 8, 128, 4, 5000), (1, 1, 1, 64, 4, 30011),
                                               (32, 8, 8, 128, 8, 1300), (1, 32, 16, 256, 4, 950), (6, 14, 2, 256, 8, 700)])
def test_weights_of_every_plan(B, Hq, Hkv, D, bits, n):
    """The one-CTA-per-SM layout, several waves in the longest-first order, one run."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    torch.manual_seed(n)
    c = tq.KVCache(B, Hkv, D, -(-n // 16) * 16, bits=bits)
    k = torch.randn((B, Hkv, n, D), device="cuda").half()
    tq.tq_quantize_kv_append(c, k, torch.randn_like(k), torch.zeros(B, dtype=torch.int32, device="cuda"))
    q = torch.randn((B, Hq, D), device="cuda").half()
    lens = np.random.default_rng(n).integers(1, n + 1, B).astype(np.int32)
    lens[0] = n
    w = torch.zeros((B, Hkv, c.capacity), device="cuda")
    out = tq.tq_sdpa_decode_weights(c, q, dev(torch, lens), n, 1 / math.sqrt(D), w, tq.weights_workspace(B, Hq, Hkv, D, n))
    G = Hq // Hkv
    rows = 2 if n > 50000 else Hkv  # heads compared in fp64 on the host
    code = {}
    for kv in "kv":
        a = getattr(c, kv + "_codes")[:, :rows]
        a = torch.stack((a & 15, a >> 4), -1).flatten(-2) if bits == 4 else a
        s, z = (getattr(c, kv + x)[:, :rows].double().repeat_interleave(64, -1) for x in ("_scale", "_bias"))
        code[kv] = (s * a.double() + z).cpu().numpy()
    qh, got_o, got_w = q.double().cpu().numpy(), host(out), w.cpu().numpy()
    for b in range(B):
        for h in range(rows):
            o, p = softmax_rows(qh[b, h * G:(h + 1) * G], code["k"][b, h, : lens[b]], code["v"][b, h, : lens[b]], 1 / math.sqrt(D))
            assert_close(got_o[b, h * G:(h + 1) * G], o)
            assert np.linalg.norm(got_w[b, h, : lens[b]] - p.sum(0)) <= 1e-5 * np.linalg.norm(p.sum(0))
            assert not got_w[b, h, lens[b]:].any()


@pytest.mark.parametrize("flags", [1, 2, 3])
def test_weights_of_a_rotated_cache(flags):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, n = 2, 10, 2, 128, 700
    c = make_cache(tq, torch, B, Hkv, D, n, 4, seed=flags, flags=flags)
    q = np.random.default_rng(3).standard_normal((B, Hq, D)).astype(np.float16)
    lens = np.array([n, 333], np.int32)
    w = torch.zeros((B, Hkv, c.capacity), device="cuda")
    qt = dev(torch, q)
    out = tq.tq_sdpa_decode_weights(c, qt, dev(torch, lens), n, 0.09, w, tq.weights_workspace(B, Hq, Hkv, D, n), flags=flags)
    q_in = host(tq.tq_hadamard_rotate(qt)) if flags & tq.TQ_ROTATE_K else q
    want_o, want_w = reference(c, q_in, lens, 0.09, np.zeros(w.shape, np.float32), 1.0)
    if flags & tq.TQ_ROTATE_V:
        H = np.array([[1.0]])
        while H.shape[0] < D:
            H = np.block([[H, H], [H, -H]])
        want_o = want_o @ H / math.sqrt(D)
    assert_close(host(out), want_o)
    check(w.cpu().numpy(), want_w, lens, Hq // Hkv)


def test_weights_lengths_outside_are_clamped_and_reported():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, n = 3, 8, 1, 128, 300
    c = make_cache(tq, torch, B, Hkv, D, n, 4, seed=5)
    q = np.random.default_rng(5).standard_normal((B, Hq, D)).astype(np.float16)
    old = np.zeros((B, Hkv, c.capacity), np.float32)
    w, st = dev(torch, old), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tq.tq_sdpa_decode_weights(c, dev(torch, q), dev(torch, np.array([999, -4, 256], np.int32)), 256, 0.09, w,
                                    tq.weights_workspace(B, Hq, Hkv, D, 256), status=st)
    want_o, want_w = reference(c, q, [256, 0, 256], 0.09, old, 1.0)
    assert_close(host(out), want_o)
    check(w.cpu().numpy(), want_w, [256, 0, 256], Hq)
    assert int(st) == tq.TQ_DEV_SEQ_LEN


def test_weights_accumulate_in_a_graph_and_on_two_streams():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, n = 2, 16, 2, 128, 3000
    c = make_cache(tq, torch, B, Hkv, D, n, 4, seed=6)
    rng = np.random.default_rng(6)
    qs = [rng.standard_normal((B, Hq, D)).astype(np.float16) for _ in range(3)]
    lens = np.array([n, 1234], np.int32)
    lt = dev(torch, lens)
    qt, out = dev(torch, qs[0]), torch.zeros((B, Hq, D), dtype=torch.float16, device="cuda")
    w, ws = torch.zeros((B, Hkv, c.capacity), device="cuda"), tq.weights_workspace(B, Hq, Hkv, D, n)
    tq.tq_sdpa_decode_weights(c, qt, lt, n, 0.09, w, ws, out=out)  # loads the kernels
    torch.cuda.synchronize()
    w.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_sdpa_decode_weights(c, qt, lt, n, 0.09, w, ws, out=out, decay=0.5)
    want = np.zeros(w.shape)
    for q in qs:
        qt.copy_(dev(torch, q))
        g.replay()
        torch.cuda.synchronize()
        want_o, want = reference(c, q, lens, 0.09, want, 0.5)
        assert_close(host(out), want_o)
    check(w.cpu().numpy(), want, lens, Hq // Hkv)
    streams, state = [torch.cuda.Stream() for _ in range(2)], []
    for q in qs[:2]:
        state.append((dev(torch, q), torch.zeros_like(w), tq.weights_workspace(B, Hq, Hkv, D, n), torch.zeros_like(out)))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (x, y, z, o) in zip(streams, state):
            tq.tq_sdpa_decode_weights(c, x, lt, n, 0.09, y, z, out=o, decay=0.0, stream=s)
    torch.cuda.synchronize()
    for q, (x, y, z, o) in zip(qs, state):
        want_o, want = reference(c, q, lens, 0.09, np.zeros(w.shape), 0.0)
        assert_close(host(o), want_o)
        check(y.cpu().numpy(), want, lens, Hq // Hkv)
