"""The chunk kernel's failure path without a GPU fault: its copying warps stop on
the way, so that the waits of all its other warps run out.  The kernel has to
record it and end, with nothing in flight, and the context, the workspace and the
cache have to serve the next call as ever."""
import math

import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import make_cache
from tests.test_gpu_chunk import queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("copies", [0, 1, 2, 5, 12])
@pytest.mark.parametrize("D,bits,Hkv,G,n,L", [(128, 4, 1, 8, 300, 2000), (64, 8, 2, 4, 5, 9000), (256, 4, 1, 2, 100, 2000), (128, 8, 2, 2, 20, 20000),
                                            (128, 4, 160, 1, 200, 1500), (64, 4, 160, 2, 30, 1500), (256, 8, 160, 1, 100, 1500)])
def test_waits_run_out_and_report(D, bits, Hkv, G, n, L, copies):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    limit_us = 3000
    c = make_cache(tq, torch, 1, Hkv, D, L, bits, seed=D + n)
    q = queries(torch, (1, Hkv * G, n, D), n)
    lens, ws = torch.tensor([L], dtype=torch.int32, device="cuda"), tq.chunk_workspace(1, Hkv * G, Hkv, D, n, L)
    scale = 1 / math.sqrt(D)
    want = tq.tq_sdpa_chunk(c, q, lens, L, scale, ws)
    out, st = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    # with all copies it is the call itself
    tq.tq_chunk_timeout_selftest(c, q, lens, L, scale, 100000, 2 ** 31 - 1, ws, out, st)
    assert torch.equal(out, want) and int(st) == 0
    e0.record()
    tq.tq_chunk_timeout_selftest(c, q, lens, L, scale, limit_us, copies, ws, out, st)
    e1.record()
    torch.cuda.synchronize()
    assert int(st) in (0, tq.TQ_DEV_TIMEOUT)
    if copies < 2:  # (a CTA has two copies at least; how many more is the plan's)
        assert int(st) == tq.TQ_DEV_TIMEOUT
    if int(st):
        assert limit_us <= e0.elapsed_time(e1) * 1e3 < 1e6
    for _ in range(2):
        st.zero_()
        assert torch.equal(tq.tq_sdpa_chunk(c, q, lens, L, scale, ws, status=st), want) and int(st) == 0
