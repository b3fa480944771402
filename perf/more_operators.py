"""The operators for several query rows and for the pages of a cache as measured
cases: attention of a chunk of new tokens over an int4 or int8 cache, cross
attention over an encoder's states held in one, and the keeping of a page pool
(forks of sequences with their pages, reservation with copy on write, compaction).

``run(state)`` is one pass through an operator: in elementary torch operations,
or, where ``own`` is true, through this library's entry points.  The caches are
the library's: codes with an fp16 scale and bias per group of 64.
"""
import math

import torch

own = False

GROUP = 64
DEV = "cuda"
ARRAYS = ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias")


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # eight drafted tokens checked against 131,072 cached ones
        dict(name="chunk 8 of 128k", op="chunk", batch=1, hq=64, hkv=8, d=128, bits=4, n=8, ragged=False, lo=131072, hi=131072, window=0, paged=False),
        # a whole prompt, causal
        dict(name="chunk prompt 8k", op="chunk", batch=1, hq=64, hkv=8, d=128, bits=4, n=8192, ragged=False, lo=8192, hi=8192, window=0, paged=False),
        # one piece of a long prompt that is taken in pieces
        dict(name="chunk 2k of 64k paged", op="chunk", batch=1, hq=64, hkv=8, d=128, bits=4, n=2048, ragged=False, lo=65536, hi=65536, window=0, paged=True),
        # a serving batch: sequences with 1 to 256 new tokens each over 1,024 to 8,192
        dict(name="chunk ragged x32 paged int8", op="chunk", batch=32, hq=64, hkv=8, d=128, bits=8, n=256, ragged=True, lo=1024, hi=8192, window=0, paged=True),
        # a prompt in a layer of wide heads that sees the last 1,024 tokens
        dict(name="chunk window 4k d256", op="chunk", batch=1, hq=32, hkv=16, d=256, bits=4, n=4096, ragged=False, lo=4096, hi=4096, window=1024, paged=False),
        # a short question after a short dialogue: latency alone
        dict(name="chunk 17 of 950 d256", op="chunk", batch=1, hq=32, hkv=16, d=256, bits=4, n=17, ragged=False, lo=950, hi=950, window=0, paged=False),
        # decoder prompts over an encoder's states of other lengths
        dict(name="cross 448 over 1500 x16", op="cross", batch=16, hq=16, hkv=16, d=64, bits=8, n=448, ragged=False, lo=311, hi=1500, window=0, paged=False),
        # the same decoders' single tokens
        dict(name="cross one token x16", op="cross", batch=16, hq=16, hkv=16, d=64, bits=8, n=1, ragged=False, lo=311, hi=1500, window=0, paged=False),
        # a step of beam search: 8 requests with 4 beams each, the beams' tail pages forked
        dict(name="fork 8 x 4 beams", op="fork", groups=8, beams=4, hkv=8, d=128, bits=4, page=128, lo=700, hi=8000, new=1),
        # 64 answers drawn from one prompt of 32,768 tokens and some
        dict(name="fork 64 answers of one prompt", op="fork", groups=1, beams=64, hkv=8, d=128, bits=8, page=256, lo=32900, hi=32900, new=16),
        # a pool half of whose pages were freed, here and there
        dict(name="compact 4096 pages", op="compact", pages=4096, live=0.5, hkv=8, d=128, bits=4, page=128, batch=32),
        # a small pool with a few holes
        dict(name="compact 96 pages", op="compact", pages=96, live=0.8, hkv=4, d=64, bits=8, page=128, batch=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "cross", "fork", "compact"])
    d = rng.choice([64, 128, 128, 256])
    hkv, bits = rng.choice([1, 2, 4, 8, 16]), rng.choice([4, 8])
    if op == "fork":
        groups, beams = _log(rng, 1, 16), rng.choice([2, 3, 4, 5, 8, 16])
        hi = _log(rng, 20, 16000)
        return dict(op="fork", groups=groups, beams=beams, hkv=hkv, d=d, bits=bits, page=rng.choice([128, 256]), lo=max(1, int(hi * rng.choice([1.0, 0.3]))), hi=hi,
                    new=rng.choice([1, 1, 4, 33, 200]))
    if op == "compact":
        most = 4096 * 8 * 128 * 4 // (hkv * d * bits)
        return dict(op="compact", pages=min(most, _log(rng, 24, 4096)), live=rng.choice([0.1, 0.3, 0.5, 0.7, 0.9]), hkv=hkv, d=d, bits=bits, page=128, batch=_log(rng, 1, 48))
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    batch = _log(rng, 1, 24)
    hi = _log(rng, 16, 65536)
    hi = max(16, min(hi, 65536 * 8 * 128 * 4 // (batch * hkv * d * bits)))
    # no more products than the largest listed case has
    most = 2048 * 65536 * 64 * 128 // (batch * hkv * group * d * hi)
    n = max(1, min(_log(rng, 1, 4096), most))
    if op == "chunk":
        n = min(n, hi)
    lo = max(1, int(hi * rng.choice([1.0, 0.5, 0.1])))
    window = _log(rng, 1, hi) if op == "chunk" and rng.random() < 0.3 else 0
    return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, bits=bits, n=n, ragged=op == "chunk" and rng.random() < 0.4, lo=lo, hi=hi, window=window,
                paged=rng.random() < 0.4)


# ------------------------------------------------------------------ the inputs
def _steps(count, lo, hi):
    return [hi] if count == 1 else [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _lengths(case):
    """(lengths, new rows) of every sequence: even steps, whatever the seed; a chunk's length counts its new rows."""
    lens = _steps(case["batch"], case["lo"], case["hi"])
    rows = _steps(case["batch"], 1, case["n"])[::-1] if case["ragged"] else [case["n"]] * case["batch"]
    if case["op"] == "chunk":
        lens = [max(a, r) for a, r in zip(lens, rows)]
    return lens, rows


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
            x.scatter_(3, at, x.gather(3, at) * 10)
        arrays = _quantize(x, case["bits"])
        del x
        if case["paged"]:
            pages = capacity // 128
            table = out.setdefault("table", torch.randperm(b * pages, generator=gen, device=DEV).to(torch.int32).view(b, pages))
            at = table.long().flatten()
            arrays = [torch.empty_like(a.view(b * pages, h, 128, -1)).index_copy_(0, at, a.unflatten(2, (pages, 128)).transpose(1, 2).reshape(b * pages, h, 128, -1)) for a in arrays]
        out.update(zip((kv + "_codes", kv + "_scale", kv + "_bias"), arrays))
    return out


def _handle(s, batch, page, pages, capacity, paged):
    """This library's cache over the state's arrays (which become the cache's own)."""
    import int4_kv_cache_gb300 as tq

    if paged:
        c = tq.PagedKVCache(batch, s["hkv"], s["d"], page, pages, s["table"].shape[1], bits=s["bits"])
        c.block_table.copy_(s["table"])
        s["table"] = c.block_table
    else:
        c = tq.KVCache(batch, s["hkv"], s["d"], capacity, bits=s["bits"])
    for name in ARRAYS:
        getattr(c, name).copy_(s[name])
        s[name] = getattr(c, name)
    return c


def _pool(s, gen, pages):
    """A pool of random pages."""
    h, p, d, bits = s["hkv"], s["page"], s["d"], s["bits"]
    for kv in "kv":
        s[kv + "_codes"] = torch.randint(0, 256, (pages, h, p, d * bits // 8), generator=gen, device=DEV, dtype=torch.uint8)
        for x in ("_scale", "_bias"):
            s[kv + x] = torch.randn((pages, h, p, d // GROUP), generator=gen, device=DEV).half()


def _prepare_fork(s, gen):
    """Beams that share their prompt's pages and have written some of their own."""
    groups, beams, page = s["groups"], s["beams"], s["page"]
    batch = groups * beams
    rows, held, pages = [], [], 0
    for n in _steps(groups, s["lo"], s["hi"]):
        total, shared = -(-n // page), (n - n // 8) // page
        prompt = list(range(pages, pages + shared))
        pages += shared
        for _ in range(beams):
            rows.append(prompt + list(range(pages, pages + total - shared)))
            pages += total - shared
            held.append(total)
    width = max(held) + (s["new"] + page - 1) // page + 1
    grow = batch * ((s["new"] + page - 1) // page + 1)
    num = pages + grow
    order = torch.randperm(num, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int64)
    for b, r in enumerate(rows):
        table[b, :len(r)] = torch.tensor(r, dtype=torch.int64)
    table = table.to(DEV)
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0)].long(), table).to(torch.int32).contiguous()
    s["held"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor([n for n in _steps(groups, s["lo"], s["hi"]) for _ in range(beams)], dtype=torch.int32, device=DEV)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=num).to(torch.int32)
    # half of each request's beams go on, each once or twice; those that end take over what another one holds
    order = torch.rand((groups, beams), generator=gen, device=DEV).argsort(1)
    go_on = (beams + 1) // 2
    pick = torch.empty_like(order).scatter_(1, order, torch.cat((order[:, :go_on], order[:, :beams - go_on]), 1))
    s["sources"] = (pick + torch.arange(groups, device=DEV).unsqueeze(1) * beams).to(torch.int32).flatten().contiguous()
    _pool(s, gen, num)
    s["num_pages"], s["batch"] = num, batch


def _prepare_compact(s, gen):
    num, batch = s["pages"], s["batch"]
    live = max(1, int(num * s["live"]))
    used = torch.randperm(num, generator=gen, device=DEV)[:live].to(torch.int32)
    # every live page once, and a first page that all sequences share
    width = -(-live // batch) + 1
    table = torch.full((batch * (width - 1),), -1, dtype=torch.int32, device=DEV)
    table[:live] = used
    table = table.view(width - 1, batch).t()
    shared = used[:1].expand(batch).unsqueeze(1)
    s["table"] = torch.cat((shared, table[:, :width - 1]), 1).contiguous()
    s["held"] = (s["table"] >= 0).sum(1).to(torch.int32)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=num).to(torch.int32)
    s["new_table"], s["new_refs"] = torch.zeros_like(s["table"]), torch.zeros_like(s["refs"])
    s["n_live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    _pool(s, gen, num)
    s["num_pages"] = num


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("fork", "compact"):
        _prepare_fork(s, gen) if case["op"] == "fork" else _prepare_compact(s, gen)
        if own:
            import int4_kv_cache_gb300 as tq

            s["cache"] = _handle(s, s["batch"], case["page"], s["num_pages"], 0, True)
            s["ws"] = tq.pages_workspace(s["cache"])
        return s
    b, d, n = case["batch"], case["d"], case["n"]
    lens, rows = _lengths(case)
    s["max_len"] = max(lens)
    s["cap"] = -(-s["max_len"] // 128) * 128 if case["paged"] else -(-s["max_len"] // 16) * 16
    order = torch.randperm(b, generator=gen, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)[order].contiguous()
    s["q_lens"] = torch.tensor(rows, dtype=torch.int32, device=DEV)[order].contiguous() if case["ragged"] else None
    s.update(_cache(case, gen, s["cap"]))
    if own:
        import int4_kv_cache_gb300 as tq

        s["cache"] = _handle(s, b, 128, b * s["cap"] // 128, s["cap"], case["paged"])
        s["ws"] = tq.chunk_workspace(b, case["hq"], case["hkv"], d, n, s["max_len"])
    s["q"] = torch.randn((b, case["hq"], n, d), generator=gen, device=DEV).half()
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.zeros((b, n, case["hq"], d), dtype=torch.float16, device=DEV)
    return s


# -------------------------------------------------------------- the plain forms
def _cached(s, kv, head, heads, n):
    """scale * code + bias in 32 bits of the first n rows of some heads: [B, heads, n, D]."""
    out = []
    for x in ("_codes", "_scale", "_bias"):
        a = s[kv + x][:, head:head + heads]
        if "table" in s:
            a = a[s["table"][:, :-(-n // 128)].long()].transpose(1, 2).flatten(2, 3)
        out.append(a[:, :, :n])
    codes, scale, bias = out
    if s["bits"] == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    g = codes.float().unflatten(-1, (-1, GROUP))
    return (g * scale.float().unsqueeze(-1) + bias.float().unsqueeze(-1)).flatten(-2)


def _plain_attention(s):
    b, h, d, n, most = s["batch"], s["hkv"], s["d"], s["n"], s["max_len"]
    group = s["hq"] // h
    lens = s["lens"].view(-1, 1, 1)
    rows = s["q_lens"].view(-1, 1, 1) if s["ragged"] else torch.full_like(lens, n)
    i, t = torch.arange(n, device=DEV).view(1, -1, 1), torch.arange(most, device=DEV).view(1, 1, -1)
    if s["op"] == "cross":
        seen = (t < lens).expand(b, n, most)
    else:
        at = lens - rows + i  # where row i stands
        seen = (t <= at) & (t < lens)
        if s["window"]:
            seen = seen & (t > at - s["window"])
    hidden = ~seen.unsqueeze(1).unsqueeze(2)
    step = max(1, min(h, (1 << 30) // (b * group * n * most)))
    for head in range(0, h, step):
        k, v = _cached(s, "k", head, min(step, h - head), most), _cached(s, "v", head, min(step, h - head), most)
        q = s["q"][:, head * group:(head + k.shape[1]) * group].float().unflatten(1, (k.shape[1], group))
        score = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (group, n)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        m = score.amax(-1, keepdim=True)
        p = score.sub_(torch.where(torch.isfinite(m), m, torch.zeros_like(m))).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p.flatten(2, 3) @ v).unflatten(2, (group, n)) / torch.where(total > 0, total, torch.ones_like(total))
        o = o.flatten(1, 2).transpose(1, 2).half()  # [B, n, heads, D]
        to = s["out"][:, :, head * group:head * group + o.shape[2]]
        to.copy_(torch.where((i < rows).unsqueeze(3), o, to))
    return s["out"]


def _plain_fork(s):
    table, held, refs = s["table"], s["held"], s["refs"]
    j = torch.arange(table.shape[1], device=DEV).view(1, -1)

    def count(t, n):
        return torch.zeros_like(refs).index_add_(0, torch.where(j < n.unsqueeze(1), t, torch.zeros_like(t)).flatten().long(),
                                                 (j < n.unsqueeze(1)).flatten().to(torch.int32))

    src = s["sources"].long()
    new_held = held[src]
    new = torch.where(j < new_held.unsqueeze(1), table[src], torch.full_like(table, -1))
    refs.add_(count(new, new_held) - count(table, held))
    table.copy_(new)
    held.copy_(new_held)
    s["lens"].copy_(s["lens"][src])
    # pages for the next rows: new ones behind the held ones, copies of shared ones that would be written
    page, start = s["page"], s["lens"].long().unsqueeze(1)
    first, last = start // page, (start + s["new"] - 1) // page
    grown = (j >= held.unsqueeze(1)) & (j <= last)
    at = table.clamp(min=0).long()
    written = (j >= first) & (j <= last) & (j < held.unsqueeze(1)) & (refs[at] > 1)
    writers = torch.zeros_like(refs).index_add_(0, at.flatten(), written.flatten().to(torch.int32))
    b = torch.arange(s["batch"], device=DEV, dtype=torch.int32).unsqueeze(1).expand_as(table)
    latest = torch.full_like(refs, -1).index_reduce_(0, at.flatten(), torch.where(written, b, torch.full_like(b, -1)).flatten(), "amax")
    copied = written & ~((writers[at] == refs[at]) & (latest[at] == b))
    wants = grown | copied
    rank = wants.flatten().cumsum(0).view_as(table) - 1
    free = torch.sort(torch.where(refs == 0, torch.arange(s["num_pages"], device=DEV), s["num_pages"])).values
    fits = wants.sum() <= (refs == 0).sum()
    got = torch.where(wants & fits, free[rank.clamp(min=0, max=s["num_pages"] - 1)], table.long()).clamp(max=s["num_pages"] - 1)
    # a candidate for a copy is the first written page of each sequence or one behind it; the others stand in for it
    width = (s["new"] + page - 2) // page + 1
    cand = (first + torch.arange(width, device=DEV)).clamp(max=table.shape[1] - 1)
    moved = (copied & fits).gather(1, cand)
    src_page = torch.where(moved, at.gather(1, cand), at.gather(1, cand[:, :1]))
    dst_page = torch.where(moved, got.gather(1, cand), got.gather(1, cand[:, :1]).clamp(min=0))
    valid = torch.where(moved, start - cand * page, start - first * page).clamp(min=0, max=page)
    src_page, dst_page = src_page.flatten(), dst_page.flatten()
    keep = (torch.arange(page, device=DEV).view(1, 1, -1, 1) < valid.view(-1, 1, 1, 1))
    for name in ARRAYS:
        a = s[name]
        a[dst_page] = torch.where(keep, a[src_page], a[dst_page])
    one = torch.ones_like(table).flatten()
    zero = torch.zeros_like(one)
    refs.index_add_(0, at.flatten(), torch.where((copied & fits).flatten(), -one, zero))
    refs.index_add_(0, got.clamp(min=0).flatten(), torch.where((wants & fits).flatten(), one, zero))
    table.copy_(got)
    held.copy_(torch.where(fits, torch.maximum(held, last.squeeze(1) + 1), held))
    return tuple(s[name] for name in ARRAYS) + (table, held, refs, s["lens"])


def _plain_compact(s):
    refs, num = s["refs"], s["num_pages"]
    live = refs > 0
    n = live.sum()
    i = torch.arange(num, device=DEV)
    src = (live & (i >= n)).nonzero().squeeze(1)
    dst = (~live & (i < n)).nonzero().squeeze(1)
    for name in ARRAYS:
        s[name][dst] = s[name][src]
    to = i.clone()
    to[src] = dst
    t = s["table"]
    s["new_table"].copy_(torch.where(torch.arange(t.shape[1], device=DEV) < s["held"].unsqueeze(1), to[t.clamp(min=0).long()].to(torch.int32), t))
    s["new_refs"].copy_(refs)
    s["new_refs"][src] = 0
    s["new_refs"][dst] = refs[src]
    s["n_live"].copy_(n)
    return tuple(s[name] for name in ARRAYS) + (s["new_table"], s["new_refs"], s["n_live"])


def run(state):
    s = state
    if own:
        import int4_kv_cache_gb300 as tq

        if s["op"] == "fork":
            tq.tq_pages_fork(s["cache"], s["refs"], s["held"], s["sources"], s["ws"], lens=s["lens"])
            tq.tq_pages_reserve(s["cache"], s["refs"], s["held"], s["lens"], s["new"], s["ws"])
            return tuple(s[name] for name in ARRAYS) + (s["table"], s["held"], s["refs"], s["lens"])
        if s["op"] == "compact":
            tq.tq_pages_compact(s["cache"], s["refs"], s["held"], s["ws"], s["new_table"], s["new_refs"], s["n_live"])
            return tuple(s[name] for name in ARRAYS) + (s["new_table"], s["new_refs"], s["n_live"])
        return tq.tq_sdpa_chunk(s["cache"], s["q"], s["lens"], s["max_len"], s["scale"], s["ws"], out=s["out"], q_lens=s["q_lens"], window=s["window"],
                                flags=tq.TQ_CHUNK_FULL if s["op"] == "cross" else 0)
    if s["op"] == "fork":
        return _plain_fork(s)
    return _plain_compact(s) if s["op"] == "compact" else _plain_attention(s)


# --------------------------------------------------------- the work of one pass
def work(case):
    h, d, bits = case["hkv"], case["d"], case["bits"]
    half = d * bits // 8 + 4 * (d // GROUP)  # a token's keys or values in one head
    if case["op"] == "fork":
        # the tables, counts and lists once in and out; the rows of the tail page of every beam that goes on twice
        batch, page = case["groups"] * case["beams"], case["page"]
        groups = _steps(case["groups"], case["lo"], case["hi"])
        entries = case["beams"] * sum(-(-n // page) for n in groups)
        rows = sum(n % page * (case["beams"] // 2) for n in groups)
        return {"bytes": 8 * entries + 16 * batch + rows * h * 4 * half, "flops": entries}
    if case["op"] == "compact":
        num = case["pages"]
        live = max(1, int(num * case["live"]))
        moved = live * (num - live) // num  # of the live pages, those that lie behind the first `live` ones
        return {"bytes": moved * case["page"] * h * 4 * half + 8 * num + 8 * (live + case["batch"]), "flops": num}
    lens, rows = _lengths(case)
    pairs, tokens = 0, 0
    for n, r in zip(lens, rows):
        if case["op"] == "cross":
            pairs += r * n
            tokens += n
            continue
        first = n - r  # the first row's position
        w = case["window"] or n
        pairs += sum(min(p + 1, w) for p in range(first, n))
        tokens += n - max(0, first - w + 1)
    return {"bytes": h * tokens * 2 * half + 4 * sum(rows) * case["hq"] * d, "flops": 4 * case["hq"] * d * pairs}


# ------------------------------------------------- from the definition, 64 bits
def _exact_rows(s, kv, b, h, n):
    """fp64 rows [n, D] of one head of sequence b."""
    parts = []
    for x in ("_codes", "_scale", "_bias"):
        a = s[kv + x]
        parts.append(torch.cat([a[p, h] for p in s["table"][b].tolist()], 0)[:n] if "table" in s else a[b, h, :n])
    codes, scale, bias = parts
    if s["bits"] == 4:
        full = torch.empty((n, s["d"]), dtype=torch.uint8, device=DEV)
        full[:, 0::2], full[:, 1::2] = codes % 16, codes // 16
        codes = full
    return scale.double().repeat_interleave(GROUP, -1) * codes.double() + bias.double().repeat_interleave(GROUP, -1)


def _exact_attention(case, s):
    lens, group = s["lens"].tolist(), case["hq"] // case["hkv"]
    rows = s["q_lens"].tolist() if case["ragged"] else [case["n"]] * case["batch"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b, (n, r) in enumerate(zip(lens, rows)):
        for h in range(case["hkv"]):
            k, v = _exact_rows(s, "k", b, h, n), _exact_rows(s, "v", b, h, n)
            for lo in range(0, r, 1024):
                hi = min(r, lo + 1024)
                stop = n if case["op"] == "cross" else n - r + hi  # no row of these sees a later token
                begin = max(0, n - r + lo - case["window"] + 1) if case["window"] else 0
                q = s["q"][b, h * group:(h + 1) * group, lo:hi].double()
                score = torch.einsum("gid,td->git", q, k[begin:stop]) * s["scale"]
                if case["op"] == "chunk":
                    age = torch.arange(n - r + lo, n - r + hi, device=DEV).unsqueeze(1) - torch.arange(begin, stop, device=DEV)
                    bad = age < 0
                    if case["window"]:
                        bad |= age >= case["window"]
                    score.masked_fill_(bad, -math.inf)
                out[b, lo:hi, h * group:(h + 1) * group] = torch.einsum("git,td->igd", torch.softmax(score, -1), v[begin:stop])
    return out


def _exact_fork(case, s):
    page, new = case["page"], case["new"]
    table, held, lens, refs = (s[k].tolist() for k in ("table", "held", "lens", "refs"))
    src = s["sources"].tolist()
    for b in range(len(table)):
        for p in table[b][:held[b]]:
            refs[p] -= 1
    width = len(table[0])
    table = [table[a][:held[a]] + [-1] * (width - held[a]) for a in src]
    held, lens = [held[a] for a in src], [lens[a] for a in src]
    for row, n in zip(table, held):
        for p in row[:n]:
            refs[p] += 1
    # each page that several write: its writers in order, the last keeps it if nobody else reads it
    writers = {}
    for b, n in enumerate(lens):
        for j in range(n // page, min(held[b], (n + new - 1) // page + 1)):
            if refs[table[b][j]] > 1:
                writers.setdefault(table[b][j], []).append((b, j))
    keeps = {w[-1] for p, w in writers.items() if len(w) == refs[p]}
    copies = {x for w in writers.values() for x in w} - keeps
    free = [p for p in range(len(refs)) if refs[p] == 0]
    arrays = {name: s[name].clone() for name in ARRAYS}
    want = [(b, j) for b in range(len(table)) for j in range((lens[b] + new - 1) // page + 1) if j >= held[b] or (b, j) in copies]
    if len(want) <= len(free):
        for (b, j), p in zip(want, free):
            refs[p] = 1
            if (b, j) in copies:
                old = table[b][j]
                refs[old] -= 1
                count = max(0, min(page, lens[b] - j * page))
                for name in ARRAYS:
                    arrays[name][p, :, :count] = s[name][old, :, :count]
            table[b][j] = p
        held = [max(x, (n + new - 1) // page + 1) for x, n in zip(held, lens)]
    back = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return tuple(arrays[name] for name in ARRAYS) + (back(table), back(held), back(refs), back(lens))


def _exact_compact(case, s):
    refs, table, held = s["refs"].tolist(), s["table"].tolist(), s["held"].tolist()
    n = sum(r > 0 for r in refs)
    holes = [p for p in range(n) if refs[p] == 0]
    late = [p for p in range(n, len(refs)) if refs[p] > 0]
    to = dict(zip(late, holes))
    arrays = {name: s[name].clone() for name in ARRAYS}
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
        for name in ARRAYS:
            arrays[name][b] = s[name][a]
    table = [[to.get(p, p) if j < c else p for j, p in enumerate(row)] for row, c in zip(table, held)]
    back = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return tuple(arrays[name] for name in ARRAYS) + (back(table), back(refs), back([n]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fork":
        return _exact_fork(case, s)
    return _exact_compact(case, s) if case["op"] == "compact" else _exact_attention(case, s)
