"""The operators around the decode step as measured cases: rotary positions with
several axes, sparse decode attention over selected blocks (with the bounds the
selection reads), decode attention that accumulates each token's attention
weight, and eviction by that weight.

``run(state)`` is one pass through an operator: in elementary torch operations,
or, where ``own`` is true, through this library's entry points.  The caches are
the library's: int4 or int8 codes with an fp16 scale and bias per group of 64.
"""
import math

import torch

own = False

GROUP = 64
DEV = "cuda"


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # the query and key of the token that each of 32 sequences decodes, its position in time, height and width
        dict(name="rope one token x32", op="rope", batch=32, n=1, hq=64, hkv=8, d=128, rotary=128, axes=3, pairs=False),
        # one prompt of text and image patches before its attention and its append
        dict(name="rope prompt 8k", op="rope", batch=1, n=8192, hq=64, hkv=8, d=128, rotary=128, axes=3, pairs=False),
        # the key bounds of a whole prompt that was just appended
        dict(name="bounds prompt 128k", op="bounds", batch=1, hkv=8, d=128, bits=4, lo=131072, hi=131072, whole=True, block=64, paged=False),
        # the bounds of the block that one decoded token of each of 32 sequences falls into
        dict(name="bounds one token x32", op="bounds", batch=32, hkv=8, d=128, bits=8, lo=1024, hi=8192, whole=False, block=64, paged=False),
        # a decode step over 4,096 of 131,072 tokens
        dict(name="sparse 128k", op="sparse", batch=1, hq=64, hkv=8, d=128, bits=4, lo=131072, hi=131072, block=64, select=64, paged=False),
        # a serving batch of 32 sequences of 1,024 to 32,768 tokens in a page pool
        dict(name="sparse ragged x32 paged", op="sparse", batch=32, hq=64, hkv=8, d=128, bits=4, lo=1024, hi=32768, block=64, select=32, paged=True),
        # a short wide-headed sequence: latency alone
        dict(name="sparse 950 d256", op="sparse", batch=1, hq=32, hkv=16, d=256, bits=8, lo=950, hi=950, block=32, select=12, paged=False),
        # a decode step at 131,072 tokens that keeps the account of what was attended to
        dict(name="weights 128k", op="weights", batch=1, hq=64, hkv=8, d=128, bits=4, lo=131072, hi=131072, decay=1.0, paged=False),
        # the same for a short wide-headed sequence
        dict(name="weights 950 d256", op="weights", batch=1, hq=32, hkv=16, d=256, bits=4, lo=950, hi=950, decay=1.0, paged=False),
        # 16 ragged sequences in 8 bits, older steps counting less
        dict(name="weights ragged x16 int8", op="weights", batch=16, hq=64, hkv=8, d=128, bits=8, lo=1024, hi=8192, decay=0.9, paged=False),
        # a prompt of 131,072 tokens cut down to 4,096 before its decode begins
        dict(name="evict 128k to 4k", op="evict", batch=1, hkv=8, d=128, bits=4, lo=131072, hi=131072, keep=4096, recent=256),
        # the budget of 32 decoding sequences restored after some hundred tokens each
        dict(name="evict 4k budget x32", op="evict", batch=32, hkv=8, d=128, bits=4, lo=4224, hi=4608, keep=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "bounds", "sparse", "sparse", "weights", "weights", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "rope":
        batch = _log(rng, 1, 32)
        n = _log(rng, 1, max(1, 8192 * 72 * 128 // (batch * hkv * (group + 1) * d)))
        axes = rng.choice([1, 2, 3, 4])
        rotary = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
        return dict(op="rope", batch=batch, n=min(n, 20000), hq=hkv * group, hkv=hkv, d=d, rotary=rotary, axes=axes, pairs=rng.random() < 0.5)
    bits, paged = rng.choice([4, 8]), rng.random() < 0.3
    batch = _log(rng, 1, 32)
    most = 131072 * 8 * 128 // (batch * hkv * d * (bits // 4))  # no more cached bytes than the largest listed case
    hi = max(2, min(_log(rng, 16, 131072), most))
    lo = max(1, int(hi * rng.choice([1.0, 0.5, 0.1])))
    if op == "bounds":
        return dict(op="bounds", batch=batch, hkv=hkv, d=d, bits=bits, lo=lo, hi=hi, whole=rng.random() < 0.6, block=rng.choice([32, 64, 128]), paged=paged)
    if op == "sparse":
        block = rng.choice([32, 64, 128])
        return dict(op="sparse", batch=batch, hq=hkv * group, hkv=hkv, d=d, bits=bits, lo=lo, hi=hi, block=block, select=_log(rng, 2, 64), paged=paged)
    if op == "weights":
        return dict(op="weights", batch=batch, hq=hkv * group, hkv=hkv, d=d, bits=bits, lo=lo, hi=hi, decay=rng.choice([1.0, 0.95, 0.5, 0.0]), paged=paged)
    keep = max(1, _log(rng, 1, max(2, min(hi, 4096))))
    return dict(op="evict", batch=batch, hkv=hkv, d=d, bits=bits, lo=lo, hi=hi, keep=keep, recent=rng.randint(0, keep))


# ------------------------------------------------------------------ the inputs
def _lengths(case):
    """The lengths of a batch: even steps from lo to hi (a seed only orders them)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi] if b == 1 else [lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _capacity(n, block):
    return -(-n // block) * block


def _quantize(x, bits):
    """fp16 rows [..., D] -> (codes, scale, bias) as the cache holds them."""
    levels = (1 << bits) - 1
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    scale, bias = ((hi - lo) / levels).half(), lo.half()
    s = scale.float().unsqueeze(-1)
    codes = torch.where(s > 0, ((g - bias.float().unsqueeze(-1)) / s).round().clamp_(0, levels), torch.zeros_like(s))
    codes = codes.to(torch.uint8).flatten(-2)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, scale, bias


def _cache(case, gen, capacity):
    """K and V of every sequence, keys with one outlier channel per head, quantized.
    Paged: the same rows in pages of 128 tokens, shuffled over the pool."""
    b, h, d = case["batch"], case["hkv"], case["d"]
    out = {}
    for kv in "kv":
        x = torch.randn((b, h, capacity, d), generator=gen, device=DEV).half()
        if kv == "k":
            at = torch.randint(0, d, (1, h, 1, 1), generator=gen, device=DEV).expand(b, h, capacity, 1)
            x.scatter_(3, at, x.gather(3, at) * 20)
        arrays = _quantize(x, case["bits"])
        del x
        if case["paged"]:
            pages = capacity // 128
            table = out.setdefault("table", torch.randperm(b * pages, generator=gen, device=DEV).to(torch.int32).view(b, pages))
            at = table.long().flatten()
            arrays = [torch.empty_like(a.view(b * pages, h, 128, -1)).index_copy_(0, at, a.unflatten(2, (pages, 128)).transpose(1, 2).reshape(b * pages, h, 128, -1)) for a in arrays]
        out.update(zip((kv + "_codes", kv + "_scale", kv + "_bias"), arrays))
    return out


def _handle(case, arrays, capacity):
    import int4_kv_cache_gb300 as tq

    if "table" in arrays:
        pages = capacity // 128
        c = tq.PagedKVCache(case["batch"], case["hkv"], case["d"], 128, case["batch"] * pages, pages, bits=case["bits"])
        c.block_table.copy_(arrays["table"])
    else:
        c = tq.KVCache(case["batch"], case["hkv"], case["d"], capacity, bits=case["bits"])
    for name in ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias"):
        getattr(c, name).copy_(arrays[name])
    return c


def _sections(case):
    half, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [half]
    first = half // 4 if axes > 2 else half // 2
    rest, parts = half - first, axes - 1
    return [first] + [rest * (i + 1) // parts - rest * i // parts for i in range(parts)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    op, b, d = case["op"], case["batch"], case["d"]
    if op == "rope":
        n, heads = case["n"], case["hq"] + 2 * case["hkv"]
        s["qkv"] = torch.randn((b, n, heads, d), generator=gen, device=DEV).half()  # one projection's rows
        s["q"], s["k"] = s["qkv"][:, :, :case["hq"]], s["qkv"][:, :, case["hq"]:case["hq"] + case["hkv"]]
        # runs of text (every axis counts on) and patches (a time step, rows and columns), far into a sequence
        t = torch.arange(n, device=DEV)
        base = torch.randint(0, 131072, (b, 1), generator=gen, device=DEV)
        axes = [base + t // 64, base + (t // 8) % 8, base + t % 8, base + t]
        s["positions"] = torch.stack((axes[3:] + axes[:3])[:case["axes"]]).to(torch.int32).contiguous()
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64) / case["rotary"])).float().to(DEV)
        s["sections"] = _sections(case)
        return s
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    s["lens"] = lens[torch.randperm(b, generator=gen, device=DEV)].contiguous()
    s["max_len"] = case["hi"]
    if op == "evict":
        paged = dict(case, paged=False)
        s["cap"] = _capacity(case["hi"], 16)
        s.update(_cache(paged, gen, s["cap"]))
        # a few tokens hold most of the weight, some were never attended to
        w = torch.exp(2.0 * torch.randn((b, case["hkv"], s["cap"]), generator=gen, device=DEV))
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.05, torch.zeros_like(w), w)
        s["dst_cap"] = _capacity(case["keep"] + 128, 16)
        shape = (b, case["hkv"], s["dst_cap"])
        s["dst"] = {k: torch.zeros(shape + (s[k].shape[3],), dtype=s[k].dtype, device=DEV) for k in ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias")}
        if own:
            s["cache"], s["to"] = _handle(paged, s, s["cap"]), _handle(paged, s["dst"], s["dst_cap"])
        s["dst_weights"] = torch.zeros(shape, device=DEV)
        s["dst_lens"] = torch.zeros(b, dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros((b, case["hkv"], case["keep"]), dtype=torch.int32, device=DEV)
        return s
    s["cap"] = _capacity(case["hi"], 128)
    s.update(_cache(case, gen, s["cap"]))
    if own:
        s["cache"] = _handle(case, s, s["cap"])
    if op == "bounds":
        nb = -(-s["cap"] // case["block"])
        s["bounds"] = torch.zeros((b, case["hkv"], nb, 2, d), dtype=torch.float16, device=DEV)
        s["n_new"] = case["lo"] if case["whole"] else 1
        s["start"] = torch.zeros_like(s["lens"]) if case["whole"] else s["lens"] - 1
        return s
    s["q"] = torch.randn((b, case["hq"], d), generator=gen, device=DEV).half()
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.zeros_like(s["q"])
    if op == "sparse":
        s["bounds"] = torch.zeros((b, case["hkv"], s["cap"] // case["block"], 2, d), dtype=torch.float16, device=DEV)
        _plain_bounds(s, s["bounds"], torch.zeros_like(s["lens"]), s["lens"], s["cap"] // case["block"])
        s["blocks"] = torch.zeros((b, case["hkv"], case["select"]), dtype=torch.int32, device=DEV)
        s["first"], s["last"] = 1 if case["select"] > 1 else 0, 1
        if own:
            import int4_kv_cache_gb300 as tq

            s["ws"] = tq.sparse_workspace(b, case["hq"], case["hkv"], d, s["max_len"], case["select"], case["block"])
    else:
        # what some twenty earlier steps have left
        s["weights"] = torch.rand((b, case["hkv"], s["cap"]), generator=gen, device=DEV) * (40.0 * case["hq"] / case["hkv"] / s["max_len"])
        if own:
            import int4_kv_cache_gb300 as tq

            s["ws"] = tq.weights_workspace(b, case["hq"], case["hkv"], d, s["max_len"])
    return s


# -------------------------------------------------------------- the plain forms
def _rows(s, name, n):
    """The first n rows of every (sequence, head) of a cache array: [B, H, n, W]."""
    a = s[name]
    if "table" in s:
        pages = -(-n // 128)
        a = a[s["table"][:, :pages].long()].transpose(1, 2).flatten(2, 3)
    return a[:, :, :n]


def _values(codes, scale, bias, bits):
    """scale * code + bias in 32 bits."""
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    g = codes.float().unflatten(-1, (-1, GROUP))
    return (g * scale.float().unsqueeze(-1) + bias.float().unsqueeze(-1)).flatten(-2)


def _cached(s, kv, n):
    return _values(_rows(s, kv + "_codes", n), _rows(s, kv + "_scale", n), _rows(s, kv + "_bias", n), s["bits"])


def _at(s, row):
    """Where logical rows [B, H, n] lie in the cache arrays."""
    ib, ih = torch.arange(s["batch"], device=DEV).view(-1, 1, 1), torch.arange(s["hkv"], device=DEV).view(1, -1, 1)
    return (s["table"].long()[ib, row // 128], ih, row % 128) if "table" in s else (ib, ih, row)


def _gathered(s, kv, row):
    at = _at(s, row)
    return _values(s[kv + "_codes"][at], s[kv + "_scale"][at], s[kv + "_bias"][at], s["bits"])


def _plain_bounds(s, bounds, start, stop, count):
    """The `count` blocks from the one that holds row `start`: the least and the greatest key of each one's rows below stop, channel by channel."""
    block, h = s["block"], s["hkv"]
    ids = (start // block).long().view(-1, 1, 1) + torch.arange(count, device=DEV)
    t = ids.unsqueeze(3) * block + torch.arange(block, device=DEV)  # [B, 1, count, block]
    k = _gathered(s, "k", t.flatten(2).expand(-1, h, -1)).unflatten(2, (count, block))
    inside = (t < stop.view(-1, 1, 1, 1)).unsqueeze(4)
    lo, hi = torch.where(inside, k, math.inf).amin(3), torch.where(inside, k, -math.inf).amax(3)
    new = torch.stack((lo, hi), 3).half()
    at = (torch.arange(s["batch"], device=DEV).view(-1, 1, 1), torch.arange(h, device=DEV).view(1, -1, 1), ids.expand(-1, h, -1))
    bounds[at] = torch.where((ids * block < stop.view(-1, 1, 1)).view(-1, 1, count, 1, 1), new, bounds[at])
    return bounds


def _top(score, n):
    """Indices of the n largest along the last axis, equal ones lowest index first."""
    return torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]


def _softmax_parts(scores):
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    return p, p.sum(-1, keepdim=True)


def _plain_rope(s):
    half = s["rotary"] // 2
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV), torch.tensor(s["sections"], device=DEV), output_size=half)
    angle = s["positions"].double()[axis].permute(1, 2, 0) * s["inv_freq"].double()  # [B, n, half]
    c, sn = torch.cos(angle).float().unsqueeze(2), torch.sin(angle).float().unsqueeze(2)

    def turn(x):
        x = x.float()
        r = x[..., :2 * half]
        a, b = (r[..., 0::2], r[..., 1::2]) if s["pairs"] else (r[..., :half], r[..., half:])
        u, v = a * c - b * sn, b * c + a * sn
        r = torch.stack((u, v), -1).flatten(-2) if s["pairs"] else torch.cat((u, v), -1)
        return torch.cat((r, x[..., 2 * half:]), -1).transpose(1, 2).contiguous().half()

    return turn(s["q"]), turn(s["k"])


def _plain_sparse(s):
    b, h, d, block, want = s["batch"], s["hkv"], s["d"], s["block"], s["select"]
    q = s["q"].view(b, h, -1, d)
    # an upper bound of q.k over each block: every channel at its better end (64 bits: blocks near the border)
    qd, bd = q.double(), s["bounds"].double()
    score = (qd.clamp(min=0) @ bd[:, :, :, 1].transpose(2, 3) + qd.clamp(max=0) @ bd[:, :, :, 0].transpose(2, 3)).amax(2)
    nb = (s["lens"].view(-1, 1, 1) + block - 1) // block
    i = torch.arange(score.shape[2], device=DEV).view(1, 1, -1)
    score = torch.where((i < s["first"]) | (i >= nb - s["last"]), torch.full_like(score, math.inf), score)
    score = torch.where(i < nb, score, torch.full_like(score, -math.inf))
    at = _top(score, min(want, score.shape[2]))
    at = torch.where(at < nb, at, torch.full_like(at, 1 << 30)).sort(-1).values
    at = torch.cat((at, torch.full((b, h, want - at.shape[2]), 1 << 30, device=DEV, dtype=at.dtype)), -1)
    s["blocks"].copy_(torch.where(at < (1 << 30), at, torch.full_like(at, -1)))
    # attention over the rows of these blocks
    row = (at.unsqueeze(3) * block + torch.arange(block, device=DEV)).flatten(2)
    seen = row < s["lens"].view(-1, 1, 1)
    row = torch.where(seen, row, torch.zeros_like(row))
    k, v = _gathered(s, "k", row), _gathered(s, "v", row)
    scores = (q.float() @ k.transpose(2, 3)) * s["scale"]
    p, total = _softmax_parts(scores.masked_fill(~seen.unsqueeze(2), -math.inf))
    out = p @ v / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(out.view(b, -1, d))
    return s["out"], s["blocks"]


def _plain_weights(s):
    b, h, d, n = s["batch"], s["hkv"], s["d"], s["max_len"]
    q = s["q"].view(b, h, -1, d).float()
    seen = torch.arange(n, device=DEV).view(1, 1, -1) < s["lens"].view(-1, 1, 1)
    scores = (q @ _cached(s, "k", n).transpose(2, 3)) * s["scale"]
    p, total = _softmax_parts(scores.masked_fill(~seen.unsqueeze(2), -math.inf))
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_((p @ _cached(s, "v", n)).view(b, -1, d))
    w = s["weights"][:, :, :n]
    w.copy_(torch.where(seen, s["decay"] * w + p.sum(2), w))
    return s["out"], s["weights"]


def _plain_evict(s):
    keep, recent, n = s["keep"], s["recent"], s["max_len"]
    lens = s["lens"].view(-1, 1, 1)
    i = torch.arange(n, device=DEV).view(1, 1, -1)
    w = torch.where(i >= lens - recent, math.inf, s["weights"][:, :, :n])
    w = torch.where(i < lens, w, -math.inf)
    at = _top(w, min(keep, n))
    at = torch.cat((at, torch.full(at.shape[:2] + (keep - at.shape[2],), n, device=DEV, dtype=at.dtype)), -1)
    at = torch.where(at < lens, at, torch.full_like(at, 1 << 30)).sort(-1).values
    full = at < (1 << 30)
    src = torch.where(full, at, torch.zeros_like(at)).unsqueeze(3)
    for name, dst in s["dst"].items():
        rows = s[name].gather(2, src.expand(-1, -1, -1, dst.shape[3]))
        dst[:, :, :keep] = torch.where(full.unsqueeze(3), rows, dst[:, :, :keep])
    s["dst_weights"].zero_()
    s["dst_weights"][:, :, :keep] = torch.where(full, s["weights"].gather(2, src.squeeze(3)), torch.zeros_like(w[..., :1]))
    s["dst_lens"].copy_(torch.clamp(s["lens"], max=keep))
    s["kept"].copy_(torch.where(full, at, torch.full_like(at, -1)))
    return dict(s["dst"], weights=s["dst_weights"], lens=s["dst_lens"], kept=s["kept"])


def run(state):
    s, op = state, state["op"]
    if own:
        import int4_kv_cache_gb300 as tq

        if op == "rope":
            return tq.tq_rope_axes(s["q"], s["k"], s["positions"], s["inv_freq"], s["sections"], flags=tq.TQ_ROPE_PAIRS if s["pairs"] else 0)
        if op == "bounds":
            return tq.tq_kv_block_bounds(s["cache"], s["bounds"], s["start"], s["n_new"], block_tokens=s["block"])
        if op == "sparse":
            return tq.tq_sparse_decode(s["cache"], s["bounds"], s["q"], s["lens"], s["max_len"], s["scale"], s["ws"], out=s["out"],
                                       blocks=s["blocks"], block_tokens=s["block"], n_first=s["first"], n_last=s["last"])
        if op == "weights":
            out = tq.tq_sdpa_decode_weights(s["cache"], s["q"], s["lens"], s["max_len"], s["scale"], s["weights"], s["ws"], out=s["out"],
                                            decay=s["decay"])
            return out, s["weights"]
        tq.tq_kv_evict(s["cache"], s["to"], s["weights"], s["lens"], s["max_len"], s["keep"], s["recent"], s["dst_weights"], s["dst_lens"],
                       s["kept"])
        to = s["to"]
        return {"k_codes": to.k_codes, "k_scale": to.k_scale, "k_bias": to.k_bias, "v_codes": to.v_codes, "v_scale": to.v_scale,
                "v_bias": to.v_bias, "weights": s["dst_weights"], "lens": s["dst_lens"], "kept": s["kept"]}
    if op == "rope":
        return _plain_rope(s)
    if op == "bounds":
        return _plain_bounds(s, s["bounds"], s["start"], s["start"] + s["n_new"], -(-s["n_new"] // s["block"]))
    if op == "sparse":
        return _plain_sparse(s)
    if op == "weights":
        return _plain_weights(s)
    return _plain_evict(s)


# --------------------------------------------------------- the work of one pass
def work(case):
    b, d = case["batch"], case["d"]
    if case["op"] == "rope":
        rows = b * case["n"] * (case["hq"] + case["hkv"])
        return {"bytes": rows * d * 4 + b * case["n"] * case["axes"] * 4 + case["rotary"] * 2, "flops": rows * case["rotary"] * 3}
    h, bits, lens = case["hkv"], case["bits"], _lengths(case)
    half = d * bits // 8 + 4 * (d // GROUP)  # a token's keys or values in one head
    if case["op"] == "bounds":
        if case["whole"]:
            rows, blocks = [case["lo"]] * b, [-(-case["lo"] // case["block"])] * b
        else:
            rows, blocks = [(n - 1) % case["block"] + 1 for n in lens], [1] * b
        return {"bytes": h * (sum(rows) * half + sum(blocks) * 4 * d), "flops": h * sum(rows) * d * 4}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": h * (sum(lens) * 4 + kept * (4 * half + 4) + b * (_capacity(case["keep"] + 128, 16) + case["keep"]) * 4), "flops": h * sum(lens)}
    hq = case["hq"]
    io = b * hq * d * 4
    if case["op"] == "weights":
        return {"bytes": h * sum(lens) * (2 * half + 8) + io, "flops": hq * sum(lens) * (4 * d + 8)}
    blocks = [-(-n // case["block"]) for n in lens]
    rows = sum(n if k <= case["select"] else case["select"] * case["block"] for n, k in zip(lens, blocks))
    scored = sum(k for k in blocks if k > case["select"])
    return {"bytes": h * (scored * 4 * d + rows * 2 * half + b * case["select"] * 4) + io, "flops": hq * (scored * 4 * d + rows * 4 * d)}


# ------------------------------------------------- from the definition, 64 bits
def _exact_kv(s, kv, b, rows=None):
    """fp64 rows [H, n, D] of sequence b (all of them, or rows [H, n])."""
    out = []
    for x in ("_codes", "_scale", "_bias"):
        a = s[kv + x]
        if "table" in s:
            a = torch.cat([a[p] for p in s["table"][b].tolist()], 1)
        else:
            a = a[b]
        if rows is not None:
            a = torch.stack([a[h][rows[h]] for h in range(a.shape[0])])
        out.append(a)
    codes, scale, bias = out
    if s["bits"] == 4:
        full = torch.empty(codes.shape[:-1] + (s["d"],), dtype=torch.uint8, device=DEV)
        full[..., 0::2] = codes % 16
        full[..., 1::2] = codes // 16
        codes = full
    spread = lambda t: t.double().repeat_interleave(GROUP, -1)  # noqa: E731
    return spread(scale) * codes.double() + spread(bias)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        both = []
        lead, freq = [], s["inv_freq"].double()
        for a, count in enumerate(s["sections"]):
            lead += [a] * count
        pos = torch.stack([s["positions"][a].double() for a in lead], -1)
        z = torch.polar(torch.ones_like(pos), pos * freq).unsqueeze(2)
        r = case["rotary"]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if case["pairs"]:
                t = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * z
                y[..., 0:r:2], y[..., 1:r:2] = t.real, t.imag
            else:
                t = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
                y[..., :r // 2], y[..., r // 2:r] = t.real, t.imag
            both.append(y.transpose(1, 2).contiguous())
        return tuple(both)
    lens = s["lens"].tolist()
    if op == "bounds":
        out = s["bounds"].double().clone()
        for b in range(case["batch"]):
            start, stop = int(s["start"][b]), int(s["start"][b]) + s["n_new"]
            k, blk = _exact_kv(s, "k", b), case["block"]
            first, last = start // blk, -(-stop // blk)
            pad = last * blk - stop
            k = torch.cat((k[:, first * blk:stop], k[:, stop - 1:stop].expand(-1, pad, -1)), 1).unflatten(1, (-1, blk))
            out[b, :, first:last, 0], out[b, :, first:last, 1] = k.min(2).values, k.max(2).values
        return out
    if op == "evict":
        dst = {k: torch.zeros_like(v) for k, v in s["dst"].items()}
        kept, dw = torch.full_like(s["kept"], -1), torch.zeros_like(s["dst_weights"])
        for b, n in enumerate(lens):
            old = max(0, min(n, n - case["recent"]))
            free = min(n, case["keep"]) - (n - old)
            for h in range(case["hkv"]):
                order = torch.argsort(-s["weights"][b, h, :old].double(), stable=True)[:free]
                rows = torch.cat((order.sort().values, torch.arange(old, n, device=DEV)))
                kept[b, h, :len(rows)] = rows.to(torch.int32)
                dw[b, h, :len(rows)] = s["weights"][b, h, rows]
                for k in dst:
                    dst[k][b, h, :len(rows)] = s[k][b, h, rows]
        dl = torch.tensor([min(n, case["keep"]) for n in lens], dtype=torch.int32, device=DEV)
        return dict(dst, weights=dw.double(), lens=dl, kept=kept)
    b_n, h_n, d = case["batch"], case["hkv"], case["d"]
    q = s["q"].double().view(b_n, h_n, -1, d)
    out = torch.zeros((b_n, case["hq"], d), dtype=torch.float64, device=DEV)
    if op == "weights":
        w = s["weights"].double().clone()
        for b, n in enumerate(lens):
            k, v = _exact_kv(s, "k", b)[:, :n], _exact_kv(s, "v", b)[:, :n]
            p = torch.softmax(torch.einsum("hgd,hnd->hgn", q[b], k) * s["scale"], -1)
            out[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(-1, d)
            w[b, :, :n] = w[b, :, :n] * case["decay"] + p.sum(1)
        return out, w
    blocks = torch.full_like(s["blocks"], -1)
    for b, n in enumerate(lens):
        blk, nb = case["block"], -(-n // case["block"])
        lo, hi = s["bounds"][b, :, :nb, 0].double(), s["bounds"][b, :, :nb, 1].double()
        chosen = []
        for h in range(h_n):
            if nb <= case["select"]:
                pick = torch.arange(nb, device=DEV)
            else:
                u = torch.maximum(q[b, h].unsqueeze(1) * lo[h], q[b, h].unsqueeze(1) * hi[h]).sum(-1).amax(0)
                mid = torch.argsort(-u[s["first"]:nb - s["last"]], stable=True)[:case["select"] - s["first"] - s["last"]] + s["first"]
                pick = torch.cat((torch.arange(s["first"], device=DEV), mid.sort().values, torch.arange(nb - s["last"], nb, device=DEV)))
            blocks[b, h, :len(pick)] = pick.to(torch.int32)
            rows = (pick.unsqueeze(1) * blk + torch.arange(blk, device=DEV)).flatten()
            chosen.append(rows[rows < n])
        k, v = _exact_kv(s, "k", b, chosen), _exact_kv(s, "v", b, chosen)
        p = torch.softmax(torch.einsum("hgd,hnd->hgn", q[b], k) * s["scale"], -1)
        out[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(-1, d)
    return out, blocks
