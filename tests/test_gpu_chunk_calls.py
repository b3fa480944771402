"""Calls of the chunk attention that its documentation allows and a first reading may
miss: workspaces with anything in them, two calls at once, one row of some sequences,
captured calls over one cache, tiles that end with a cache, long windows.  Tolerances
as in test_gpu_chunk.py."""
import math

import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache
from tests.test_gpu_chunk import attend, check, queries, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,L,D,Hkv", [(4, 20000, 128, 1), (300, 3000, 64, 2), (40, 9000, 256, 1)])
def test_workspace_holds_anything(n, L, D, Hkv):
    """Partial states are written before they are read."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 2, Hkv, D, L, seed=n)
    q = queries(torch, (2, 4 * Hkv, n, D), n)
    lens = torch.tensor([L, 100], dtype=torch.int32, device="cuda")
    ws = tq.chunk_workspace(2, 4 * Hkv, Hkv, D, n, L)
    outs = []
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        outs.append(tq.tq_sdpa_chunk(c, q, lens, L, 0.1, ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check(torch, outs[0], reference(torch, c, q, [L, 100], [n, n], 0.1), [n, n])


def test_two_calls_at_once():
    """Two streams, a workspace each, one cache."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    L, n = 6000, 64
    c = make_cache(tq, torch, 1, 4, 128, L, seed=2)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    qs = [queries(torch, (1, 16, n, 128), s) for s in (1, 2)]
    ws = [tq.chunk_workspace(1, 16, 4, 128, n, L) for _ in qs]
    want = [tq.tq_sdpa_chunk(c, q, lens, L, 0.1, w) for q, w in zip(qs, ws)]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[torch.empty_like(want[0]) for _ in range(6)] for _ in qs]
    torch.cuda.synchronize()
    for i in range(6):
        for s, st in enumerate(streams):
            tq.tq_sdpa_chunk(c, qs[s], lens, L, 0.1, ws[s], out=outs[s][i], stream=st)
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(o, want[s]) for o in outs[s])


@pytest.mark.parametrize("full", [False, True])
def test_single_rows_of_some_sequences(full):
    """n = 1 with row counts: sequences without a row keep their output."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens, rows = [900, 30, 0, 411], [1, 0, 1, 1]
    c = make_cache(tq, torch, 4, 2, 128, 900, seed=3)
    q = queries(torch, (4, 16, 1, 128), 4)
    out = torch.full((4, 1, 16, 128), 3.0, dtype=torch.float16, device="cuda")
    attend(torch, tq, c, q, lens, rows, full=full, out=out)
    assert bool((out[1] == 3.0).all()) and not bool(out[2].any())
    check(torch, out, reference(torch, c, q, lens, rows, 1 / math.sqrt(128), full=full), rows)


@pytest.mark.parametrize("L", [16, 128, 144, 257, 400])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 8), (256, 4), (256, 8)])
def test_tiles_that_end_with_the_cache(D, bits, L):
    """Caches whose last tile is cut off by their end (rows behind it are not theirs)."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    cap = -(-L // 16) * 16
    c = make_cache(tq, torch, 2, 2, D, L, bits, seed=L, capacity=cap)
    q = queries(torch, (2, 4, 20, D), L)
    check(torch, attend(torch, tq, c, q, [L, max(1, L - 9)]), reference(torch, c, q, [L, max(1, L - 9)], [20, 20], 1 / math.sqrt(D)), [20, 20])


def test_windows_past_the_length():
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 1, 2, 128, 700, seed=5)
    q = queries(torch, (1, 8, 90, 128), 6)
    want = attend(torch, tq, c, q, [700])
    assert torch.equal(attend(torch, tq, c, q, [700], window=2 ** 31 - 1), want)


@pytest.mark.parametrize("Hkv,G,n,L", [(2, 8, 1000, 4000), (40, 2, 520, 700)])
def test_some_items_whole_others_cut(Hkv, G, n, L):
    """More items than SMs, and some left over: the last ones are cut into runs."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 4, Hkv, 128, L, seed=7)
    q = queries(torch, (4, Hkv * G, n, 128), 8)
    lens = [L, L, L - 5, n]
    check(torch, attend(torch, tq, c, q, lens, flags=0), reference(torch, c, q, lens, [n] * 4, 1 / math.sqrt(128)), [n] * 4)


def test_steep_scores():
    """Maxima that grow from tile to tile by more than the rescaling leaves alone, and rows far below others."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    for D in (64, 128, 256):
        c = make_cache(tq, torch, 1, 1, D, 1500, seed=9, outliers=False)
        # keys that grow along the sequence: later tiles win
        grow = torch.linspace(0.1, 3.0, c.capacity, device="cuda").half().view(1, 1, -1, 1)
        c.k_scale.mul_(grow)
        c.k_bias.mul_(grow)
        q = queries(torch, (1, 4, 200, D), 10)
        for scale in (0.5, -0.5):
            got = attend(torch, tq, c, q, [1500], scale=scale)
            check(torch, got, reference(torch, c, q, [1500], [200], scale), [200])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_one_row_either_way(D, bits, paged):
    """One row a sequence is the decode, with row counts it is not: the same rows, zeros and reports."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    lens = [500, 0, 1, 700, -3]  # the last two: past max_seq_len, below none
    held = [500, 0, 1, 512, 0]
    c = make_cache(tq, torch, 5, 2, D, 512, bits, paged, seed=D)
    q = queries(torch, (5, 8, 1, D), 11)
    for scale in (1 / math.sqrt(D), -0.05):
        for full in (False, True):
            ref = reference(torch, c, q, held, [1] * 5, scale, full=full)
            for rows in (None, [1] * 5):
                st = torch.zeros(1, dtype=torch.int32, device="cuda")
                out = attend(torch, tq, c, q, lens, rows, full=full, scale=scale, max_len=512, status=st)
                check(torch, out, ref, [1] * 5)
                assert int(st) == tq.TQ_DEV_SEQ_LEN and not bool(out[1].any()) and not bool(out[4].any())


def test_binding_refusals():
    """What the binding refuses before the library is called."""
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    c = make_cache(tq, torch, 2, 2, 64, 64, seed=1)
    q = queries(torch, (2, 4, 8, 64), 1)
    lens = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    ws = tq.chunk_workspace(2, 4, 2, 64, 8, 64)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(2, 3)), dict(q=q[..., :32]), dict(q=q[0]), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long()),
               dict(q_lens=lens[:1]), dict(workspace=ws.float()), dict(out=torch.empty_like(q)), dict(status=lens.long()), dict(seq_lens=lens.cpu())):
        a = dict(dict(cache=c, q=q, seq_lens=lens, max_seq_len=64, attn_scale=1.0, workspace=ws), **kw)
        with pytest.raises(ValueError):
            tq.tq_sdpa_chunk(**a)
    with pytest.raises(tq.TQError):
        tq.tq_sdpa_chunk(c, q, lens, 65, 1.0, ws)
    with pytest.raises(tq.TQError):
        tq.tq_sdpa_chunk(c, q, lens, 64, 1.0, ws[:256])
    with pytest.raises(ValueError):
        tq.chunk_workspace(2, 5, 2, 64, 8, 64)
    refs, held = lens.clone(), lens.clone()
    with pytest.raises(ValueError):
        tq.tq_pages_fork(c, refs, held, lens, ws)  # not a paged cache
    p = tq.PagedKVCache(2, 2, 64, 128, 5, 3)
    refs, held = tq.page_state(p)
    pw = tq.pages_workspace(p)
    for call in (lambda: tq.tq_pages_fork(p, held, held, lens, pw), lambda: tq.tq_pages_reserve(p, refs, held, lens[:1], 1, pw),
                 lambda: tq.tq_pages_compact(p, refs, held, pw, p.block_table[:1], refs, lens[:1])):
        with pytest.raises(ValueError):
            call()
