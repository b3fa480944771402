"""fp64 references for the entry points around the decode step, from the cache
arrays' stored codes (elementary operations; no library kernel)."""
import numpy as np


def rows(cache, name):
    """A cache array in logical order [B, Hkv, capacity, W] (host numpy)."""
    a = getattr(cache, name).cpu().numpy()
    if not getattr(cache, "paged", False):
        return a
    table = cache.block_table.cpu().numpy()
    g = a[table].transpose(0, 2, 1, 3, 4)  # [B, Hkv, pages, page_tokens, W]
    return g.reshape(g.shape[0], g.shape[1], -1, g.shape[4])


def values(cache, kv):
    """fp64 scale * code + bias [B, Hkv, capacity, D] (exact: 8 + 11 bits plus 11)."""
    codes = rows(cache, kv + "_codes")
    if cache.bits == 4:
        full = np.empty(codes.shape[:-1] + (cache.head_dim,), np.uint8)
        full[..., 0::2] = codes & 15
        full[..., 1::2] = codes >> 4
        codes = full
    s, z = (np.repeat(rows(cache, kv + x).astype(np.float64), 64, -1) for x in ("_scale", "_bias"))
    return s * codes.astype(np.float64) + z


def softmax_rows(q, k, v, scale):
    """fp64 (output [G, D], weights [G, n]) of queries q [G, D] over rows k, v [n, D]."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros((q.shape[0], 0))
    s = (q @ k.T) * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return p @ v, p


def make_cache(tq, torch, B, Hkv, D, n, bits=4, paged=False, seed=0, capacity=None, flags=0, outliers=True, page_tokens=128):
    """A cache holding n random rows per sequence (one outlier key channel per head)."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, Hkv, n, D)).astype(np.float32)
    v = rng.standard_normal((B, Hkv, n, D)).astype(np.float32)
    if outliers:
        for h in range(Hkv):
            k[:, h, :, rng.integers(0, D)] *= 20
    if paged:
        per = -(-(capacity or n) // page_tokens)
        c = tq.PagedKVCache(B, Hkv, D, page_tokens, B * per + 2, per, bits=bits)
        c.buffer.zero_()
        c.block_table.copy_(torch.from_numpy(rng.permutation(B * per + 2)[: B * per].astype(np.int32).reshape(B, per)))
    else:
        c = tq.KVCache(B, Hkv, D, capacity or max(16, -(-n // 16) * 16), bits=bits)
        c.buffer.zero_()
    if n:
        tq.tq_quantize_kv_append(c, torch.from_numpy(k.astype(np.float16)).cuda(), torch.from_numpy(v.astype(np.float16)).cuda(),
                                 torch.zeros(B, dtype=torch.int32, device="cuda"), flags=flags)
    return c


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.dtype.is_floating_point else t.cpu().numpy()
