"""The entry points around the decode step on a cache whose arrays pass 2^32
bytes: the last kv head of the second sequence lies past it.  References in
fp64 with torch on the device, over that head's rows alone."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import assert_close, need_gpu
from tests.operator_helpers import dev, host

pytestmark = pytest.mark.gpu

B, HKV, HQ, D, CAP = 2, 8, 16, 128, (1 << 22) + 4096


@pytest.fixture(scope="module")
def big():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = tq.KVCache(B, HKV, D, CAP)
    assert c.k_codes.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in (c.k_codes, c.v_codes):
        a.view(torch.int64).random_(generator=g)
    for kv in "kv":
        getattr(c, kv + "_scale").uniform_(0.1, 0.3, generator=g)
        getattr(c, kv + "_bias").uniform_(-2.5, -1.0, generator=g)
    yield torch, tq, c
    del c
    torch.cuda.empty_cache()


def head_values(torch, c, kv, b, h, rows):
    """fp64 rows (a slice or an index) of one head, on the device."""
    codes = getattr(c, kv + "_codes")[b, h][rows]
    codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s, z = (getattr(c, kv + x)[b, h][rows].double().repeat_interleave(64, -1) for x in ("_scale", "_bias"))
    return s * codes.double() + z


def test_bounds_and_listed_blocks(big):
    torch, tq, c = big
    bounds = tq.block_bounds(c, 128)
    start = CAP - 300
    tq.tq_kv_block_bounds(c, bounds, dev(torch, np.array([0, start], np.int32)), 300, block_tokens=128)
    blocks = torch.tensor([CAP // 128 - 1, 3, CAP // 128 - 200, -1], dtype=torch.int32, device="cuda").expand(B, HKV, 4).contiguous()
    q = torch.randn((B, HQ, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).half()
    lens = dev(torch, np.array([CAP, CAP - 5], np.int32))
    ws = tq.sparse_workspace(B, HQ, HKV, D, CAP, 4, 128)
    out = tq.tq_sdpa_blocks_decode(c, q, blocks, lens, CAP, 1 / math.sqrt(D), ws, block_tokens=128)
    b, h = B - 1, HKV - 1
    for j in (start // 128, CAP // 128 - 1):
        k = head_values(torch, c, "k", b, h, slice(j * 128, (j + 1) * 128)).cpu().numpy().astype(np.float16)
        got = bounds[b, h, j].cpu().numpy()
        assert np.array_equal(got[0], k.min(0)) and np.array_equal(got[1], k.max(0))
    assert not bounds[b, h, : start // 128].any()
    rows = torch.cat([torch.arange(j * 128, min((j + 1) * 128, CAP - 5), device="cuda") for j in (CAP // 128 - 1, 3, CAP // 128 - 200)])
    k, v = head_values(torch, c, "k", b, h, rows), head_values(torch, c, "v", b, h, rows)
    qh = q[b, -2:].double()
    p = torch.softmax(qh @ k.T / math.sqrt(D), -1)
    assert_close(host(out)[b, -2:], (p @ v).cpu().numpy())


def test_weights_and_eviction(big):
    torch, tq, c = big
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((B, HQ, D), device="cuda", generator=g).half()
    lens = dev(torch, np.array([1000, CAP - 77], np.int32))
    w = torch.zeros((B, HKV, CAP), device="cuda")
    ws = tq.weights_workspace(B, HQ, HKV, D, CAP)
    out = tq.tq_sdpa_decode_weights(c, q, lens, CAP, 1 / math.sqrt(D), w, ws)
    del ws
    b, h, n = B - 1, HKV - 1, CAP - 77
    k = head_values(torch, c, "k", b, h, slice(0, n))
    p = torch.softmax(q[b, -2:].double() @ k.T / math.sqrt(D), -1)
    del k
    o = p @ head_values(torch, c, "v", b, h, slice(0, n))
    assert_close(host(out)[b, -2:], o.cpu().numpy())
    want = p.sum(0)
    assert float((w[b, h, :n].double() - want).norm() / want.norm()) <= 1e-5
    assert not w[b, h, n:].any()
    keep, recent = 1000, 40
    dst = tq.KVCache(B, HKV, D, 1008)
    dw, dl = torch.zeros((B, HKV, 1008), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, HKV, keep), dtype=torch.int32, device="cuda")
    tq.tq_kv_evict(c, dst, w, lens, CAP, keep, recent, dw, dl, kept)
    order = torch.sort(w[b, h, : n - recent], descending=True, stable=True).indices[: keep - recent].sort().values
    rows = torch.cat((order, torch.arange(n - recent, n, device="cuda")))
    assert torch.equal(kept[b, h].long(), rows)
    assert torch.equal(dw[b, h, :keep], w[b, h, rows]) and dl.tolist() == [1000, keep]
    for name in ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias"):
        assert torch.equal(getattr(dst, name)[b, h, :keep], getattr(c, name)[b, h][rows]), name
