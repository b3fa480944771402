// evict.cu -- eviction from a cache by accumulated attention weight: of every
// (sequence, kv head) the last `recent` rows and, of the rows before them, the
// keep - recent of greatest weight (equal weights the lowest index first), in
// their order, into another cache.
//
// Two kernels.  select: one cluster of CTAs per (sequence, kv head), each with
// a stretch of the weights, 8 or 32 a thread in registers (longer stretches are read
// again, from L2, in every step); the threshold weight by radix selection on
// the ordered fp32 key: for its first 11 bits every CTA counts into its own
// histogram and adds what is not zero to the first CTA's, which picks the digit
// and tells the others; a cluster then gathers the keys that share it in the
// first CTA, which finds the threshold among them (one CTA, or more than kGather
// such keys: two more steps of 11 and 10 bits); then the kept rows' indices in order, from counts per warp
// and prefix sums over warps and CTAs.  copy: the kept rows, codes and
// scales, 16 bytes a thread, into consecutive rows of the destination, with
// streaming stores (32 sequences of 4,096 rows 64.1 -> 61.4 us).  Bound
// by the kept rows' bytes for a batch, by the selection's latency for one
// sequence.
#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_radix.cuh"

namespace tq {

namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;
constexpr int kGather = 4096;  // keys that the first CTA takes over
static_assert(kBins == 4 * kEvThreads && kEvThreads == 512, "four bins, one digit count a thread");

__device__ __forceinline__ uint32_t weight_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
    return (u & 0x80000000u) != 0u ? ~u : (u | 0x80000000u);
}

// V: 16-byte loads of a thread, 2,048 weights of the CTA's stretch each.  ONE:
// they cover the stretch, which is read once.
template <int V, bool ONE>
__global__ void __launch_bounds__(kEvThreads, V == 8 ? 1 : 2) evict_select_kernel(const EvictParams p) {
    constexpr int kStretch = V * 4 * kEvThreads;
    constexpr int kRoundWarps = V * kEvWarps;       // 128-weight pieces of a round
    __shared__ uint32_t hist[kBins];                // this CTA's counts
    __shared__ uint32_t sums[kBins];                // the first CTA's: the cluster's counts
    __shared__ uint32_t wcount[kEvWarps];
    __shared__ uint32_t piece[kRoundWarps];         // above (low half) and equal (high half) of each piece
    __shared__ uint32_t pick[3];
    __shared__ uint32_t found[kGather];             // the first CTA's: keys that share the first digit
    __shared__ uint32_t n_found;
    __shared__ uint32_t digits[2][256];
    __shared__ uint32_t cta_count[2];               // this CTA's rows above the threshold, and equal to it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_cta = p.ctas, rank = static_cast<int>(blockIdx.x) % n_cta;
    const int bh = static_cast<int>(blockIdx.x) / n_cta;
    const int b = bh / p.num_kv_heads;
    for (int i = threadIdx.x; i < kBins; i += kEvThreads) hist[i] = sums[i] = 0;
    digits[threadIdx.x >> 8][threadIdx.x & 255] = 0;
    if (threadIdx.x == 0) n_found = 0;
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
    const bool all = len <= p.keep;      // the whole cluster: every row stays
    const int old = len - p.recent;      // else: rows that compete, old > want
    const int want = p.keep - p.recent;  // of them stay
    const bool choose = !all && want > 0;

    // this CTA's stretch [s0, s1), in rounds of kStretch weights
    const int per = choose ? ((old + n_cta - 1) / n_cta + 3) & ~3 : 0;
    const int s0 = min(rank * per, old), s1 = min(s0 + per, old);
    float4 held[V];
    auto load_round = [&](int base) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + (v * kEvThreads + threadIdx.x) * 4;
            if (i < s1) held[v] = __ldg(reinterpret_cast<const float4*>(weights + i));
        }
    };
    // f(weight, its row) for each of this thread's weights of a round
    auto visit_round = [&](int base, auto f) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + (v * kEvThreads + threadIdx.x) * 4;
            const float w[4] = {held[v].x, held[v].y, held[v].z, held[v].w};
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (i + c < s1) f(w[c]);
        }
    };
    if (choose) load_round(s0);

    // what needs no selection
    for (int i = kept + part; i < p.out_weight_stride; i += parts) out_w[i] = 0.0f;
    for (int i = kept + part; i < p.keep; i += parts) list[i] = -1;
    if (bh % p.num_kv_heads == 0 && part == 0) p.out_lens[b] = kept;
    if (all) {
        for (int i = part; i < len; i += parts) {
            list[i] = i;
            out_w[i] = weights[i];
        }
        return;
    }
    for (int i = part; i < p.recent; i += parts) {
        list[want + i] = old + i;
        out_w[want + i] = weights[old + i];
    }
    if (!choose) return;

    if (n_cta > 1) cluster_sync();  // every CTA runs, its counts are zero
    else __syncthreads();
    uint32_t value = 0, mask = 0;
    int above = 0;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        for (int base = s0; base < s1; base += kStretch) {
            if (!ONE) load_round(base);
            visit_round(base, [&](float w) {
                const uint32_t k = weight_key(w);
                if ((k & mask) == value) atomicAdd(&hist[(k >> shift) & (bins - 1u)], 1u);
            });
            if (ONE) break;
        }
        const int top = kBins - 1 - 4 * threadIdx.x;  // this thread's four bins, largest first
        if (n_cta > 1) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t c = hist[top - j];
                if (c != 0) {
                    red_cluster_add_u32(&sums[top - j], 0, c);
                    hist[top - j] = 0;
                }
            }
            cluster_sync();
        } else {
            __syncthreads();
        }
        uint32_t* from = n_cta > 1 ? sums : hist;
        if (rank == 0) {
            uint32_t c[4], sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = from[top - j];
                from[top - j] = 0;
                sum += c[j];
            }
            uint32_t before = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += o;
            }
            if (lane == 31) wcount[warp] = before;
            __syncthreads();
            before -= sum;
            for (int w = 0; w < warp; ++w) before += wcount[w];
            const uint32_t need = static_cast<uint32_t>(want - above);
            if (before < need && need <= before + sum) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (before < need && need <= before + c[j]) {
                        for (int r = 0; r < n_cta; ++r) {
                            if (n_cta > 1) {
                                st_cluster_u32(&pick[0], r, top - j);
                                st_cluster_u32(&pick[1], r, above + before);
                                st_cluster_u32(&pick[2], r, c[j]);
                            } else {
                                pick[0] = top - j;
                                pick[1] = above + before;
                                pick[2] = c[j];
                            }
                        }
                    }
                    before += c[j];
                }
            }
        }
        if (n_cta > 1) cluster_sync();
        else __syncthreads();
        value |= pick[0] << shift;
        above = static_cast<int>(pick[1]);
        mask |= (bins - 1u) << shift;
        const uint32_t share = pick[2];
        if (pass == 0 && n_cta > 1 && share <= kGather) {  // the same for the cluster
            for (int base = s0; base < s1; base += kStretch) {
                if (!ONE) load_round(base);
                visit_round(base, [&](float w) {
                    const uint32_t k = weight_key(w);
                    if ((k & mask) != value) return;
                    st_cluster_u32(&found[min(atom_cluster_add_u32(&n_found, 0, 1), kGather - 1u)], 0, k);
                });
                if (ONE) break;
            }
            cluster_sync();
            if (rank == 0) {
                int larger;
                const uint32_t t = nth_largest<kEvThreads, uint32_t>(
                    want - above, static_cast<int>(share), value, value | ~mask,
                    [&](auto f) { for (uint32_t i = threadIdx.x; i < share; i += kEvThreads) f(found[i]); }, digits, larger);
                if (threadIdx.x < n_cta) {
                    st_cluster_u32(&pick[0], threadIdx.x, t);
                    st_cluster_u32(&pick[1], threadIdx.x, above + larger);
                }
            }
            cluster_sync();
            value = pick[0];
            above = static_cast<int>(pick[1]);
            break;
        }
        if (n_cta == 1) __syncthreads();  // pick and wcount are read before the next pass writes them
    }
    const uint32_t ties = static_cast<uint32_t>(want - above);  // rows equal to the threshold that stay, lowest index first

    // ---- the list.  Rows in order: round, then piece (v, warp) of 128, then lane, then the lane's four.
    auto counts_of = [&](int base, int v) -> uint32_t {  // of this thread's four: above | equal << 16
        const int i = base + (v * kEvThreads + threadIdx.x) * 4;
        const float w[4] = {held[v].x, held[v].y, held[v].z, held[v].w};
        uint32_t n = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (i + c < s1) {
                const uint32_t k = weight_key(w[c]);
                n += (k > value ? 1u : 0u) + (k == value ? 0x10000u : 0u);
            }
        }
        return n;
    };
    uint32_t gt = 0, eq = 0;  // above and equal before the current round
    if (n_cta > 1) {          // the CTAs before this one
        uint32_t n_gt = 0, n_eq = 0;
        for (int base = s0; base < s1; base += kStretch) {
            if (!ONE) load_round(base);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t n = counts_of(base, v);
                n_gt += n & 0xffffu;
                n_eq += n >> 16;
            }
            if (ONE) break;
        }
        if (threadIdx.x < 2) cta_count[threadIdx.x] = 0;
        __syncthreads();
        n_gt = __reduce_add_sync(0xffffffffu, n_gt);
        n_eq = __reduce_add_sync(0xffffffffu, n_eq);
        if (lane == 0) {
            atomicAdd(&cta_count[0], n_gt);
            atomicAdd(&cta_count[1], n_eq);
        }
        cluster_sync();
        uint32_t c_gt = 0, c_eq = 0;
        if (lane < rank) {
            c_gt = ld_cluster_u32(&cta_count[0], lane);
            c_eq = ld_cluster_u32(&cta_count[1], lane);
        }
        gt = __reduce_add_sync(0xffffffffu, c_gt);
        eq = __reduce_add_sync(0xffffffffu, c_eq);
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA has read the others' counts
    }
    for (int base = s0; base < s1; base += kStretch) {
        if (!ONE) load_round(base);
        uint32_t before[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t n = counts_of(base, v);
            uint32_t incl = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            before[v] = incl - n;
            if (lane == 31) piece[v * kEvWarps + warp] = incl;
        }
        __syncthreads();
        // exclusive prefix over the pieces (a round holds at most 16,384 rows: no carry between the halves)
        if (warp == 0) {
            constexpr int P = kRoundWarps / 32;
            static_assert(kRoundWarps % 32 == 0 && kStretch <= 16384, "whole lanes; counts fit 16 bits");
            uint32_t c[P], sum = 0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                c[j] = piece[lane * P + j];
                sum += c[j];
            }
            uint32_t run = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, run, off);
                if (lane >= off) run += o;
            }
            if (lane == 31) wcount[0] = run;
            run -= sum;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                piece[lane * P + j] = run;
                run += c[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + (v * kEvThreads + threadIdx.x) * 4;
            const uint32_t at0 = before[v] + piece[v * kEvWarps + warp];
            uint32_t g = gt + (at0 & 0xffffu), e = eq + (at0 >> 16);
            const float w[4] = {held[v].x, held[v].y, held[v].z, held[v].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (i + c >= s1) break;
                const uint32_t k = weight_key(w[c]);
                if (k > value || (k == value && e < ties)) {
                    const uint32_t at = g + min(e, ties);
                    list[at] = i + c;
                    out_w[at] = w[c];
                }
                g += k > value ? 1u : 0u;
                e += k == value ? 1u : 0u;
            }
        }
        gt += wcount[0] & 0xffffu;
        eq += wcount[0] >> 16;
        if (ONE) break;
        __syncthreads();
    }
    if (n_cta > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // nobody reads this CTA's memory any more
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
        if (kv < 2 && rr < n) __stcs(reinterpret_cast<uint4*>((kv ? p.dst_v : p.dst_k) + to[rr] * BPT) + c, x[j]);
    }
    if (r < n) *reinterpret_cast<Row*>(p.dst_sb[a] + to[r] * NG) = s;
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.num_kv_heads * p.ctas);
    cfg.blockDim = dim3(kEvThreads);
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
    const long long most = (static_cast<long long>(p.max_seq_len) - p.recent + p.ctas - 1) / p.ctas;  // a CTA's stretch
    using Kern = void (*)(EvictParams);
    const Kern k = most <= kEvStretch / 4 ? evict_select_kernel<2, true>
                                          : (most <= kEvStretch ? evict_select_kernel<8, true> : evict_select_kernel<8, false>);
    return cudaLaunchKernelEx(&cfg, k, p);
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
