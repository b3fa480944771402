"""Forks, reservations and compaction of a page pool against a plain Python
account of the same pages (every value is exact: whole numbers and copied rows)."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

ARRAYS = ("k_codes", "k_scale", "k_bias", "v_codes", "v_scale", "v_bias")


class Pool:
    """The plain account: lists of pages, counts, and the rows."""

    def __init__(self, cache, refs, held, lens):
        self.table, self.refs, self.held, self.lens = (t.cpu().numpy().astype(np.int64) for t in (cache.block_table, refs, held, lens))
        self.rows = {a: getattr(cache, a).cpu().numpy().copy() for a in ARRAYS}
        self.page = cache.page_tokens

    def fork(self, src):
        old, oh, ol = self.table.copy(), self.held.copy(), self.lens.copy()
        for b in range(len(src)):
            for p in old[b, :oh[b]]:
                self.refs[p] -= 1
        for b, s in enumerate(src):
            self.held[b], self.lens[b] = (oh[s], ol[s]) if s >= 0 else (0, 0)
            self.table[b] = -1
            self.table[b, :self.held[b]] = old[s, :self.held[b]]
            for p in self.table[b, :self.held[b]]:
                self.refs[p] += 1

    def reserve(self, start, n):
        spans = {b: (s // self.page, (s + n - 1) // self.page) for b, s in enumerate(start) if s >= 0 and s + n <= self.table.shape[1] * self.page}
        writers = {}
        for b, (lo, hi) in spans.items():
            for j in range(lo, min(hi + 1, self.held[b])):
                if self.refs[self.table[b, j]] > 1:
                    writers.setdefault(int(self.table[b, j]), []).append((b, j))
        copies = {x for p, w in writers.items() for x in (w[:-1] if len(w) == self.refs[p] else w)}
        want = [(b, j) for b, (lo, hi) in spans.items() for j in range(hi + 1) if (b, j) in copies or j >= self.held[b]]
        free = np.flatnonzero(self.refs == 0)
        if len(want) > len(free):
            return False
        for (b, j), p in zip(want, free):
            if (b, j) in copies:
                q = self.table[b, j]
                keep = min(self.page, max(0, start[b] - j * self.page))
                for a in ARRAYS:
                    self.rows[a][p, :, :keep] = self.rows[a][q, :, :keep]
                self.refs[q] -= 1
            self.table[b, j], self.refs[p] = p, 1
        for b, (lo, hi) in spans.items():
            self.held[b] = max(self.held[b], hi + 1)
        return True

    def compact(self):
        n = int((self.refs > 0).sum())
        to = {int(p): int(h) for p, h in zip(np.flatnonzero(self.refs > 0)[n - len(np.flatnonzero(self.refs[:n] <= 0)):] if (self.refs[:n] <= 0).any() else [],
                                             np.flatnonzero(self.refs[:n] <= 0))}
        moved = np.where(self.refs > 0, np.arange(len(self.refs)), -1)
        for p, h in to.items():
            for a in ARRAYS:
                self.rows[a][h] = self.rows[a][p]
            self.refs[h], self.refs[p], moved[p] = self.refs[p], 0, h
        for b in range(len(self.table)):
            for j in range(self.held[b]):
                self.table[b, j] = to.get(int(self.table[b, j]), self.table[b, j])
        return n, moved

    def same(self, cache, refs, held, lens):
        for name, want, got in (("table", self.table, cache.block_table), ("refs", self.refs, refs), ("held", self.held, held), ("lens", self.lens, lens)):
            assert np.array_equal(want, got.cpu().numpy()), name
        for a in ARRAYS:
            got = getattr(cache, a).cpu().numpy()
            assert np.array_equal(got.view(np.uint8), self.rows[a].view(np.uint8)), a


def pool(torch, tq, B, Hkv=2, D=64, page=128, pages=40, per=8, bits=4, seed=0):
    c = tq.PagedKVCache(B, Hkv, D, page, pages, per, bits=bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c.buffer.copy_(torch.randint(0, 256, c.buffer.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.block_table.fill_(-1)
    refs, held = tq.page_state(c)
    return c, refs, held, torch.zeros(B, dtype=torch.int32, device="cuda"), tq.pages_workspace(c)


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hkv,D,page,bits", [(2, 64, 128, 4), (8, 128, 128, 4), (1, 64, 256, 8), (3, 256, 128, 8), (5, 128, 384, 4)])
@pytest.mark.parametrize("B,per,pages", [(6, 8, 60), (1, 3, 4), (33, 300, 1500), (140, 9, 900)])
def test_a_life_of_a_pool(B, per, pages, Hkv, D, page, bits):
    """Prompts, forks, steps, ends and compaction in random order."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    if pages * Hkv * page * D > 3e8:
        pytest.skip("a large pool once is enough")
    c, refs, held, lens, ws = pool(torch, tq, B, Hkv, D, page, pages, per, bits)
    rng = np.random.default_rng(B + D)
    ref = Pool(c, refs, held, lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(14):
        what = rng.integers(0, 4) if step else 1
        if what == 0:
            src = np.where(rng.random(B) < 0.2, -1, np.where(rng.random(B) < 0.5, np.arange(B), rng.integers(0, B, B)))
            tq.tq_pages_fork(c, refs, held, i32(torch, src), ws, lens=lens, status=st)
            ref.fork(src)
        elif what == 3:
            n_live, moved = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros_like(refs)
            tq.tq_pages_compact(c, refs, held, ws, c.block_table, refs, n_live, moved=moved, status=st)
            n, m = ref.compact()
            assert int(n_live) == n and np.array_equal(moved.cpu().numpy(), m)
        else:
            n = int(rng.choice([1, 1, 7, page, 2 * page + 3]))
            start = ref.lens.copy()
            start[start + n > per * page] = -1
            tq.tq_pages_reserve(c, refs, held, i32(torch, start), n, ws, status=st)
            bits_now = (tq.TQ_DEV_WRITE_POS if (start < 0).any() else 0)
            if ref.reserve(start, n):
                ref.lens = np.where(start >= 0, start + n, ref.lens)
                lens.copy_(torch.from_numpy(ref.lens.astype(np.int32)))
            else:
                bits_now |= tq.TQ_DEV_NO_PAGE
            assert int(st) == bits_now
            st.zero_()
        assert int(st) == 0
        ref.same(c, refs, held, lens)


def test_last_writer_keeps():
    """Who copies of a page that is shared by writers and by others."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 4, pages=20)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, -1, -1, -1]), 200, ws)
    lens[0] = 200
    tq.tq_pages_fork(c, refs, held, i32(torch, [0, 0, 0, 0]), ws, lens=lens)
    assert refs[:2].tolist() == [4, 4] and lens.tolist() == [200] * 4
    ref = Pool(c, refs, held, lens)
    for start in ([200, 200, -1, 200], [-1, -1, 200, -1], [200] * 4, [128, 129, 0, 255]):
        tq.tq_pages_reserve(c, refs, held, i32(torch, start), 1, ws)
        assert ref.reserve(np.array(start), 1)
        ref.same(c, refs, held, lens)
    # a reference of the caller's own keeps the page from every writer
    refs[int(c.block_table[3, 1])] += 1
    ref = Pool(c, refs, held, lens)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [-1, -1, -1, 200]), 1, ws)
    ref.reserve(np.array([-1, -1, -1, 200]), 1)
    ref.same(c, refs, held, lens)


def test_too_few_pages():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 2, pages=5)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, 0]), 384, ws, status=st)
    assert int(st) == tq.TQ_DEV_NO_PAGE and not bool(refs.any()) and not bool(held.any()) and bool((c.block_table == -1).all())
    st.zero_()
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, -1]), 384, ws, status=st)
    assert int(st) == tq.TQ_DEV_WRITE_POS and held.tolist() == [3, 0]
    # freeing makes room
    tq.tq_pages_fork(c, refs, held, i32(torch, [-1, 1]), ws)
    assert not bool(refs.any())
    st.zero_()
    tq.tq_pages_reserve(c, refs, held, i32(torch, [-1, 0]), 640, ws, status=st)
    assert c.block_table[1, :5].tolist() == [0, 1, 2, 3, 4] and refs.tolist() == [1] * 5


def test_bad_arguments_on_the_device():
    """Sources, held counts, table entries and rows outside their ranges are reported and harm nothing."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 3, pages=20, per=4)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, 0, 0]), 300, ws)
    ref = Pool(c, refs, held, lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_pages_fork(c, refs, held, i32(torch, [3, -2, 2 ** 31 - 1]), ws, status=st)
    assert int(st) == tq.TQ_DEV_SOURCE
    ref.same(c, refs, held, lens)
    st.zero_()
    tq.tq_pages_reserve(c, refs, held, i32(torch, [-1, 4 * 128, 2 ** 31 - 1]), 1, ws, status=st)
    assert int(st) == tq.TQ_DEV_WRITE_POS
    ref.same(c, refs, held, lens)
    for call in (lambda: tq.tq_pages_fork(c, refs, held, i32(torch, [0, 1, 2]), ws, status=st),
                 lambda: tq.tq_pages_reserve(c, refs, held, i32(torch, [0, 0, 0]), 1, ws, status=st),
                 lambda: tq.tq_pages_compact(c, refs, held, ws, c.block_table, refs, torch.zeros_like(st), status=st)):
        st.zero_()
        c.block_table[1, 0] = 2 ** 31 - 1
        call()
        assert int(st) == tq.TQ_DEV_PAGE and int(c.block_table[1, 0]) == 2 ** 31 - 1
        c.block_table[1, 0] = int(ref.table[1, 0])
        refs.copy_(torch.from_numpy(ref.refs.astype(np.int32)))
    st.zero_()
    held[2] = 99
    tq.tq_pages_compact(c, refs, held, ws, torch.empty_like(c.block_table), torch.empty_like(refs), torch.zeros_like(st), status=st)
    assert int(st) == tq.TQ_DEV_PAGE


def test_compact_apart():
    """Table and counts into arrays of their own; repeated it does the same again."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 5, pages=90, per=16)
    for n in (700, 130, 400):
        tq.tq_pages_reserve(c, refs, held, lens, n, ws)
        lens += n
    tq.tq_pages_fork(c, refs, held, i32(torch, [-1, 1, 1, -1, 4]), ws, lens=lens)
    table, counts, n_live = torch.zeros_like(c.block_table), torch.full_like(refs, 9), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = (c.block_table.clone(), refs.clone())
    ref = Pool(c, refs, held, lens)
    n, _ = ref.compact()
    for _ in range(2):
        tq.tq_pages_compact(c, refs, held, ws, table, counts, n_live)
        assert torch.equal(before[0], c.block_table) and torch.equal(before[1], refs)
        assert int(n_live) == n and np.array_equal(table.cpu().numpy(), ref.table) and np.array_equal(counts.cpu().numpy(), ref.refs)
        for a in ARRAYS:
            assert np.array_equal(getattr(c, a).cpu().numpy().view(np.uint8), ref.rows[a].view(np.uint8))
    assert not bool(counts[n:].any()) and bool((counts[:n] > 0).all())


def test_nothing_in_use():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 2, pages=7)
    n_live = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    tq.tq_pages_compact(c, refs, held, ws, c.block_table, refs, n_live)
    tq.tq_pages_reserve(c, refs, held, lens, 0, ws)
    tq.tq_pages_fork(c, refs, held, i32(torch, [1, 0]), ws)
    assert int(n_live) == 0 and not bool(refs.any()) and bool((c.block_table == -1).all())


def test_captured_steps():
    """A beam step (fork, reserve) captured and replayed with new sources."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 4, pages=60)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, -1, -1, -1]), 180, ws)
    lens[0] = 180
    src = i32(torch, [0, 0, 0, 0])

    def step():
        tq.tq_pages_fork(c, refs, held, src, ws, lens=lens)
        tq.tq_pages_reserve(c, refs, held, lens, 3, ws)
        lens.add_(3)

    ref = Pool(c, refs, held, lens)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(1)
    for it in range(30):
        s = rng.integers(0, 4, 4) if it else np.zeros(4, int)
        src.copy_(torch.from_numpy(s.astype(np.int32)))
        g.replay()
        ref.fork(s)
        assert ref.reserve(ref.lens, 3)
        ref.lens += 3
    ref.same(c, refs, held, lens)


@pytest.mark.parametrize("bits,rotate", [(4, 0), (8, 3)])
def test_a_serving_loop(bits, rotate):
    """Reserve, append, chunk, fork into beams, append and decode, compact, chunk again: the beams read what caches of
    their own would hold."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    B, Hq, Hkv, D, page, per = 4, 8, 2, 128, 128, 6
    c, refs, held, lens, ws = pool(torch, tq, B, Hkv, D, page, 24, per, bits)
    own = tq.KVCache(B, Hkv, D, page * per, bits=bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    cws, dws = tq.chunk_workspace(B, Hq, Hkv, D, 300, page * per), tq.workspace(B, Hq, Hkv, D, page * per)
    rotated = dict(flags=rotate)

    def both(n, start, new_lens, q_lens=None):
        k, v, q = rnd(B, Hkv, n, D), rnd(B, Hkv, n, D), rnd(B, Hq, n, D)
        tq.tq_pages_reserve(c, refs, held, start, n, ws)
        out = []
        for cache in (c, own):
            tq.tq_quantize_kv_append(cache, k, v, start, **rotated)
            out.append(tq.tq_sdpa_chunk(cache, q, new_lens, page * per, D ** -0.5, cws, q_lens=q_lens, **rotated) if n > 1 else
                       tq.tq_sdpa_int4_decode(cache, q[:, :, 0].contiguous(), new_lens, page * per, D ** -0.5, dws, **rotated))
        a, b = out
        if q_lens is not None:
            a, b = a[:1], b[:1]
        assert float((a.double() - b.double()).norm()) <= 1e-3 * float(b.double().norm())

    start = i32(torch, [0, -1, -1, -1])
    both(300, start, i32(torch, [300, 0, 0, 0]), i32(torch, [300, 0, 0, 0]))
    lens[0] = 300
    tq.tq_pages_fork(c, refs, held, i32(torch, [0, 0, 0, 0]), ws, lens=lens)
    for a in ARRAYS:
        getattr(own, a)[1:] = getattr(own, a)[:1]
    for step in range(5):
        both(1, lens, lens + 1)
        lens += 1
        src = i32(torch, [[1, 1, 3, 3], [0, 2, 0, 2], [3, 2, 1, 0], [0, 0, 0, 0], [0, 1, 2, 3]][step])
        tq.tq_pages_fork(c, refs, held, src, ws, lens=lens)
        for a in ARRAYS:
            t = getattr(own, a)
            t.copy_(t[src.long()])
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_pages_compact(c, refs, held, ws, c.block_table, refs, n_live)
    assert int(n_live) < 24
    both(40, lens, lens + 40)


def test_pools_past_32_bits():
    """Pages whose codes lie behind 2^32 bytes."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    pages = (1 << 32) // (4 * 128 * 128) + 40  # 64 KB of codes a page
    c = tq.PagedKVCache(2, 4, 128, 128, pages, 8, bits=8)
    refs, held = tq.page_state(c)
    ws = tq.pages_workspace(c)
    refs.fill_(1)
    refs[pages - 30:] = 0  # all but the last pages are someone else's
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, -1]), 200, ws)
    assert c.block_table[0, :2].tolist() == [pages - 30, pages - 29]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = {}
    for a in ARRAYS:
        t = getattr(c, a)
        for p in (pages - 30, pages - 29):
            t[p].view(torch.uint8).copy_(torch.randint(0, 256, t[p].view(torch.uint8).shape, generator=g, device="cuda", dtype=torch.uint8))
        rows[a] = t[pages - 30:pages - 28].clone()
    # the second sequence takes both over and writes to the second
    tq.tq_pages_fork(c, refs, held, i32(torch, [0, 0]), ws)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [-1, 200]), 1, ws)
    p = int(c.block_table[1, 1])
    assert p == pages - 28 and int(c.block_table[1, 0]) == pages - 30
    for a in ARRAYS:
        assert torch.equal(getattr(c, a)[p, :, :72].view(torch.uint8), rows[a][1, :, :72].view(torch.uint8))
    # the others let go: the three move to the front
    refs[:pages - 30] = 0
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_pages_compact(c, refs, held, ws, c.block_table, refs, n_live)
    assert int(n_live) == 3 and c.block_table[:, :2].tolist() == [[0, 1], [0, 2]] and refs[:4].tolist() == [2, 1, 1, 0]
    for a in ARRAYS:
        assert torch.equal(getattr(c, a)[:2].view(torch.uint8), rows[a].view(torch.uint8))


def test_long_prompts():
    """Rows that fall into more entries than a step's."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c, refs, held, lens, ws = pool(torch, tq, 3, pages=170, per=60)  # 157 in use at most
    ref = Pool(c, refs, held, lens)
    for start, n in (([0, -1, 0], 5000), ([100, 4990, 5100], 2200), ([0, 7300, 200], 1)):
        tq.tq_pages_reserve(c, refs, held, i32(torch, start), n, ws)
        assert ref.reserve(np.array(start), n)
        ref.same(c, refs, held, lens)
    src = np.array([2, 2, 2])
    tq.tq_pages_fork(c, refs, held, i32(torch, src), ws)
    ref.fork(src)
    tq.tq_pages_reserve(c, refs, held, i32(torch, [0, 128, -1]), 4300, ws)  # whole shared prompts written over
    assert ref.reserve(np.array([0, 128, -1]), 4300)
    ref.lens = lens.cpu().numpy()
    ref.same(c, refs, held, lens)
