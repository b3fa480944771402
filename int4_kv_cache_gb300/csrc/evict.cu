// evict.cu -- eviction from a cache by accumulated attention weight: of every
// (sequence, kv head) the last `recent` rows and, of the rows before them, the
// keep - recent of greatest weight (equal weights the lowest index first), in
// their order, into another cache.
//
// Two kernels.  select: one cluster of CTAs per (sequence, kv head), each with
// a stretch of the weights (held in shared memory where they fit, else read
// again); the threshold weight by radix selection (11, 11 and 10 bits of the
// ordered fp32 key) over the cluster's histograms, then the kept rows'
// indices in order (counts per warp, prefix sums over warps and CTAs).
// copy: the kept rows, codes and scales, 16 bytes a thread, into consecutive
// rows of the destination.  Bound by the kept rows' bytes for a batch, by the
// selection's latency for one sequence.
#include <atomic>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t weight_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
    return (u & 0x80000000u) != 0u ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ float held[];  // this CTA's stretch of weights, if it fits
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wcount[2][kEvWarps];
    __shared__ int pick[2];
    __shared__ uint32_t cta_count[2];  // this CTA's rows above the threshold, and equal to it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_cta = p.ctas, rank = static_cast<int>(blockIdx.x) % n_cta;
    const int bh = static_cast<int>(blockIdx.x) / n_cta;
    const int b = bh / p.num_kv_heads;
    pdl_wait_primary();
    pdl_launch_dependents();
    int len = __ldcg(p.seq_lens + b);
    if (len < 0 || len > p.max_seq_len) {
        if (p.status != nullptr && threadIdx.x == 0 && rank == 0 && bh % p.num_kv_heads == 0)
            atomicOr(p.status, TQ_DEV_SEQ_LEN);
        len = min(max(len, 0), p.max_seq_len);
    }
    const int kept = min(len, p.keep);
    const float* weights = p.weights + static_cast<long long>(bh) * p.weight_stride;
    int32_t* list = p.kept + static_cast<long long>(bh) * p.keep;
    float* out_w = p.out_weights + static_cast<long long>(bh) * p.out_weight_stride;
    const int part = rank * kEvThreads + threadIdx.x, parts = n_cta * kEvThreads;
    for (int i = kept + part; i < p.out_weight_stride; i += parts) out_w[i] = 0.0f;
    for (int i = kept + part; i < p.keep; i += parts) list[i] = -1;
    if (bh % p.num_kv_heads == 0 && part == 0) p.out_lens[b] = kept;
    if (len <= p.keep) {  // the whole cluster: every row stays
        for (int i = part; i < len; i += parts) {
            list[i] = i;
            out_w[i] = weights[i];
        }
        return;
    }
    const int old = len - p.recent;           // rows that compete; old > want
    const int want = p.keep - p.recent;       // of them stay
    for (int i = part; i < p.recent; i += parts) {
        list[want + i] = old + i;
        out_w[want + i] = weights[old + i];
    }
    if (want == 0) return;

    // this CTA's stretch [s0, s1)
    const int per = ((old + n_cta - 1) / n_cta + 31) & ~31;
    const int s0 = min(rank * per, old), s1 = min(s0 + per, old), n = s1 - s0;
    const float* src = weights + s0;
    const bool fits = n <= p.held;
    uint32_t value = 0, mask = 0;
    int above = 0;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        for (int i = threadIdx.x; i < kBins; i += kEvThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kEvThreads) {
            float w;
            if (pass == 0) {
                w = __ldg(src + i);
                if (fits) held[i] = w;
            } else {
                w = fits ? held[i] : __ldg(src + i);
            }
            const uint32_t k = weight_key(w);
            if ((k & mask) == value) atomicAdd(&hist[(k >> shift) & (bins - 1u)], 1u);
        }
        __syncthreads();
        if (n_cta > 1) cluster_sync();
        // every CTA: thread t sums bins [base, base + 4) over the cluster, largest bins first
        uint32_t c[4], sum = 0;
        const int top = kBins - 1 - 4 * threadIdx.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = 0;
        for (int r = 0; r < n_cta; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] += n_cta > 1 ? ld_cluster_u32(&hist[top - j], r) : hist[top - j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += c[j];
        uint32_t before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += o;
        }
        if (lane == 31) wcount[0][warp] = before;
        __syncthreads();
        before -= sum;
        for (int w = 0; w < warp; ++w) before += wcount[0][w];
        const uint32_t need = static_cast<uint32_t>(want - above);
        if (before < need && need <= before + sum) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before < need && need <= before + c[j]) {
                    pick[0] = top - j;
                    pick[1] = above + static_cast<int>(before);
                }
                before += c[j];
            }
        }
        if (n_cta > 1) cluster_sync();  // also: every CTA has read this histogram
        else __syncthreads();
        value |= static_cast<uint32_t>(pick[0]) << shift;
        above = pick[1];
        mask |= (bins - 1u) << shift;
    }
    const int ties = want - above;  // rows equal to the threshold that stay, lowest index first

    // ---- the list: counts per warp (each a consecutive stretch), then places
    const int span = ((n + kEvWarps - 1) / kEvWarps + 31) & ~31;
    const int w0 = min(warp * span, n), w1 = min(w0 + span, n);
    uint32_t n_gt = 0, n_eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = weight_key(fits ? held[i] : __ldg(src + i));
        n_gt += k > value;
        n_eq += k == value;
    }
    n_gt = __reduce_add_sync(0xffffffffu, n_gt);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        wcount[0][warp] = n_gt;
        wcount[1][warp] = n_eq;
    }
    __syncthreads();
    uint32_t gt = 0, eq = 0, all_gt = 0, all_eq = 0;
#pragma unroll
    for (int w = 0; w < kEvWarps; ++w) {
        if (w < warp) {
            gt += wcount[0][w];
            eq += wcount[1][w];
        }
        all_gt += wcount[0][w];
        all_eq += wcount[1][w];
    }
    if (n_cta > 1) {
        if (threadIdx.x == 0) {
            cta_count[0] = all_gt;
            cta_count[1] = all_eq;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            gt += ld_cluster_u32(&cta_count[0], r);
            eq += ld_cluster_u32(&cta_count[1], r);
        }
        cluster_sync();  // no CTA leaves while another reads its counts
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        float w = 0.0f;
        uint32_t k = 0;
        if (i < w1) {
            w = fits ? held[i] : __ldg(src + i);
            k = weight_key(w);
        }
        const bool is_gt = i < w1 && k > value, is_eq = i < w1 && k == value;
        const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
        const uint32_t rank_eq = eq + __popc(be & below);
        const uint32_t at = gt + __popc(bg & below) + min(rank_eq, static_cast<uint32_t>(ties));
        if (is_gt || (is_eq && rank_eq < static_cast<uint32_t>(ties))) {
            list[at] = s0 + i;
            out_w[at] = w;
        }
        gt += __popc(bg);
        eq += __popc(be);
    }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;  // destination rows of a CTA

template <int BPT, int NG>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictCopyParams p) {
    __shared__ long long from[kCopyRows], to[kCopyRows];
    const int bh = blockIdx.y, b = bh / p.num_kv_heads, h = bh - b * p.num_kv_heads;
    const int r0 = blockIdx.x * kCopyRows;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int n = min(kCopyRows, min(__ldcg(p.lens + b), p.keep) - r0);
    if (n <= 0) return;
    if (threadIdx.x < n) {
        const int t = __ldcg(p.kept + static_cast<long long>(bh) * p.keep + r0 + threadIdx.x);
        from[threadIdx.x] = kv_row(p.src_map, p.num_kv_heads, b, h, t, p.status);
        to[threadIdx.x] = kv_row(p.dst_map, p.num_kv_heads, b, h, r0 + threadIdx.x, p.status);
    }
    __syncthreads();
    constexpr int PIECES = BPT / 16;
    // codes of K then V, all in flight at once
    constexpr int PER = (2 * kCopyRows * PIECES + kCopyThreads - 1) / kCopyThreads;
    uint4 x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * kCopyThreads + threadIdx.x;
        const int kv = i / (kCopyRows * PIECES), r = i / PIECES % kCopyRows, c = i % PIECES;
        if (kv < 2 && r < n)
            x[j] = __ldcs(reinterpret_cast<const uint4*>((kv ? p.src_v : p.src_k) + from[r] * BPT) + c);
    }
    struct alignas(2 * NG) Row {
        uint16_t v[NG];
    };
    const int a = threadIdx.x / kCopyRows, r = threadIdx.x % kCopyRows;  // 4 arrays x 64 rows = 256 threads
    static_assert(kCopyThreads == 4 * kCopyRows, "a thread per row of each scale and bias array");
    Row s;
    if (r < n) s = *reinterpret_cast<const Row*>(p.src_sb[a] + from[r] * NG);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * kCopyThreads + threadIdx.x;
        const int kv = i / (kCopyRows * PIECES), rr = i / PIECES % kCopyRows, c = i % PIECES;
        if (kv < 2 && rr < n) *(reinterpret_cast<uint4*>((kv ? p.dst_v : p.dst_k) + to[rr] * BPT) + c) = x[j];
    }
    if (r < n) *reinterpret_cast<Row*>(p.dst_sb[a] + to[r] * NG) = s;
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams& p, int held_bytes, cudaStream_t stream) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxEvictHeldBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.num_kv_heads * p.ctas);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(held_bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_evict_copy(const EvictCopyParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.keep + kCopyRows - 1) / kCopyRows),
                       static_cast<unsigned>(p.batch) * p.num_kv_heads);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    using Kern = void (*)(EvictCopyParams);
    Kern k = nullptr;
    switch (p.head_dim) {
        case 64: k = p.bits == 8 ? evict_copy_kernel<64, 1> : evict_copy_kernel<32, 1>; break;
        case 128: k = p.bits == 8 ? evict_copy_kernel<128, 2> : evict_copy_kernel<64, 2>; break;
        case 256: k = p.bits == 8 ? evict_copy_kernel<256, 4> : evict_copy_kernel<128, 4>; break;
        default: return cudaErrorInvalidValue;
    }
    return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace tq
