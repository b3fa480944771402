"""Outputs that a call makes on a stream other than the current one: their memory
is not memory that the current stream still uses, and is not handed out again
before the current stream is past its use of them."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.operator_helpers import dev, make_cache

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, N = 4, 32, 4, 128, 500


def calls(tq, torch):
    c = make_cache(tq, torch, B, HKV, D, N, 4, seed=3)
    q = dev(torch, np.random.default_rng(3).standard_normal((B, HQ, D)).astype(np.float16))
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    x, pos = q.view(B, 1, HQ, D), lens.view(1, B, 1).contiguous()
    inv = torch.ones(D // 2, device="cuda")
    blocks = torch.arange(4, dtype=torch.int32, device="cuda").repeat(B, HKV, 1).contiguous()
    ws, wws = tq.sparse_workspace(B, HQ, HKV, D, N, 4, 64), tq.weights_workspace(B, HQ, HKV, D, N)
    dws = tq.workspace(B, HQ, HKV, D, N)
    w = torch.zeros((B, HKV, c.capacity), device="cuda")
    return {
        "rope": lambda s: tq.tq_rope_axes(x, None, pos, inv, (D // 2,), stream=s),
        "blocks": lambda s: tq.tq_sdpa_blocks_decode(c, q, blocks, lens, N, 0.09, ws, stream=s),
        "weights": lambda s: tq.tq_sdpa_decode_weights(c, q, lens, N, 0.09, w, wws, decay=0.0, stream=s),
        "decode": lambda s: tq.tq_sdpa_int4_decode(c, q, lens, N, 0.09, dws, stream=s),
        "rotate": lambda s: tq.tq_hadamard_rotate(q, stream=s),
    }


@pytest.mark.parametrize("name", ["rope", "blocks", "weights", "decode", "rotate"])
def test_outputs_of_another_stream(name):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    call = calls(tq, torch)[name]
    want = call(None).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # memory whose last owner's reader is still queued on the current stream
    a = torch.ones_like(want)
    at = a.data_ptr()
    torch.cuda._sleep(20_000_000)
    copy = a.clone()
    del a
    out = call(side)
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert bool((copy == 1).all()) and torch.equal(out, want)
    # an output that is let go while its reader is still queued on the current stream
    at = out.data_ptr()
    torch.cuda._sleep(20_000_000)
    copy = out.clone()
    del out
    with torch.cuda.stream(side):
        other = [torch.zeros_like(want) for _ in range(4)]
    assert at not in [t.data_ptr() for t in other]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
