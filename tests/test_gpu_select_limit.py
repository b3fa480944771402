"""Selection at its limit, 22,528 blocks of a sequence, whose keys and tiles take
nearly all of an SM's shared memory: with clusters (few rows), one wide CTA a row,
and more rows than SMs.  Compared exactly with the order of fp64 scores."""
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

NB, BLOCK = 22528, 32


def reference(torch, bounds, q, lens, K, first, last):
    """The lists from fp64 scores, a row at a time (int32 [B, Hkv, K])."""
    B, H = bounds.shape[:2]
    g = q.view(B, H, -1, q.shape[-1]).double()
    out = torch.full((B, H, K), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        nb = -(-lens[b] // BLOCK)
        for h in range(H):
            lo, hi = bounds[b, h, :nb, 0].double(), bounds[b, h, :nb, 1].double()
            score = (hi @ g[b, h].clamp(min=0).T + lo @ g[b, h].clamp(max=0).T).amax(1)
            if nb <= K:
                out[b, h, :nb] = torch.arange(nb, device="cuda")
                continue
            mid = torch.sort(score[first: nb - last], descending=True, stable=True).indices[: K - first - last] + first
            out[b, h, :first] = torch.arange(first, device="cuda")
            out[b, h, first: K - last] = mid.sort().values
            out[b, h, K - last:] = torch.arange(nb - last, nb, device="cuda")
    return out


@pytest.mark.parametrize("K", [64, 5000])
@pytest.mark.parametrize("B,Hkv,G", [(1, 1, 8), (3, 8, 2), (10, 16, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_selection_of_the_most_blocks(D, B, Hkv, G, K):
    torch = need_gpu()
    import int4_kv_cache_gb300 as tq

    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + B)
    cap = NB * BLOCK
    bounds = (2 * torch.randn((B, Hkv, NB, 2, D), generator=gen, device="cuda")).half().sort(3).values.contiguous()
    bounds[:, :, 4000:9000:7] = bounds[:, :, 4001:9001:7].clone()  # equal scores
    q = torch.randn((B, Hkv * G, D), generator=gen, device="cuda").half()
    lens = [cap - 45 * b * b for b in range(B)]
    blocks = torch.full((B, Hkv, K), -7, dtype=torch.int32, device="cuda")
    ws, st = tq.sparse_workspace(B, Hkv * G, Hkv, D, cap, K, BLOCK), torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_select_blocks(bounds, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), cap, ws, blocks, cap, block_tokens=BLOCK, n_first=1,
                        n_last=2, status=st)
    assert int(st) == 0
    assert torch.equal(blocks, reference(torch, bounds, q, lens, K, 1, 2))
