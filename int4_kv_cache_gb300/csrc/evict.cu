// evict.cu -- eviction from a cache by accumulated attention weight: of every
// (sequence, kv head) the last `recent` rows and, of the rows before them, the
// keep - recent of greatest weight (equal weights the lowest index first), in
// their order, into another cache.
//
// Two kernels.  select: one cluster of CTAs per (sequence, kv head), each with
// a stretch of the weights, 8 or 16 a thread in registers (longer stretches are
// read again, from L2, in every step); the threshold weight by radix selection
// on the ordered fp32 key.  A step costs one exchange: every CTA counts its
// keys' digit into its own histogram and adds what is not zero to every CTA's
// sums, from which each finds the digit by itself.  When few enough keys share
// the digits so far, every CTA sends its own ones, and how many it has above
// them, to all, and each finds the threshold and its place in the list by
// itself.  Then the kept rows' indices in order, from counts per warp and
// prefix sums.  copy: the kept rows and their weights, codes and scales 16
// bytes a thread, into consecutive rows of the destination, with streaming
// stores; rows that stay whatever their weight (the last ones; all of a short
// sequence) are copied while the selection runs.
//
// Bound by the kept rows' bytes for a batch: 32 sequences x 8 heads, 4,096 of
// 4,608 rows each (320 MB), 62.6 us, 5.1 TB/s (pages of 128 rows: 64.7).  By the
// selection's chain of steps for one sequence: 4,096 of 131,072 rows x 8 heads
// 18.3 us (paged 18.9); 16.0 with the weights and rows in L2, 11 of them the
// selection.  (There, with one CTA that finds each digit and the threshold and
// tells the others, 19.7; the keys in shared memory instead of registers 18.2;
// 512 threads of 32 keys, whose code is twice as long and fetched once, 17.2.)
#include <atomic>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_radix.cuh"

namespace tq {

namespace {

constexpr int kBins = 2048;
constexpr int kShare = 2048;   // keys of a digit that the CTAs send each other

// A key in the order of the weights; 0 is kept for places without one.
__device__ __forceinline__ uint32_t weight_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
    return (u & 0x80000000u) != 0u ? max(~u, 1u) : (u | 0x80000000u);
}

// V: 16-byte loads of a thread.  ONE: they cover the CTA's stretch, which is
// read once.
template <int V, int THREADS, bool ONE>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const EvictParams p) {
    constexpr int kWarps = THREADS / 32;
    constexpr int kLoad = 4 * THREADS;              // weights that the CTA loads at a time
    constexpr int kRound = V * kLoad;               // and holds
    constexpr int kPieces = V * kWarps;             // of 128 weights
    constexpr int kOwnBins = kBins / THREADS;       // a thread's
    extern __shared__ uint32_t found[];             // cluster: kShare keys of each CTA
    __shared__ uint32_t hist[kBins];                // this CTA's counts
    __shared__ uint32_t sums[2][kBins];             // the cluster's counts, of even and odd steps
    __shared__ uint32_t wcount[kWarps];
    __shared__ uint32_t piece[kPieces];             // above (low half) and equal (high half) of each piece
    __shared__ uint32_t pick[3];
    __shared__ uint32_t own[2];                     // this CTA's keys above the digits so far, and those that share them
    __shared__ uint32_t above_of[8], share_of[8];   // every CTA's
    __shared__ uint32_t before_cta[2];              // rows of the CTAs before this one: above the threshold, equal to it
    __shared__ uint32_t digits[2][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_cta = p.ctas, rank = static_cast<int>(blockIdx.x) % n_cta;
    const int bh = static_cast<int>(blockIdx.x) / n_cta;
    const int b = bh / p.num_kv_heads;
    for (int i = threadIdx.x; i < kBins; i += THREADS) hist[i] = sums[0][i] = sums[1][i] = 0;
    if (threadIdx.x < 512) digits[threadIdx.x >> 8][threadIdx.x & 255] = 0;
    if (threadIdx.x < 2) own[threadIdx.x] = before_cta[threadIdx.x] = 0;
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
    const int part = rank * THREADS + threadIdx.x, parts = n_cta * THREADS;
    const bool all = len <= p.keep;      // the whole cluster: every row stays
    const int old = len - p.recent;      // else: rows that compete, old > want
    const int want = p.keep - p.recent;  // of them stay
    const bool choose = !all && want > 0;

    // this CTA's stretch [s0, s1), in rounds
    const int per = choose ? ((old + n_cta - 1) / n_cta + 3) & ~3 : 0;
    const int s0 = min(rank * per, old), s1 = min(s0 + per, old);
    float4 w[V];
    uint32_t keys[V][4];
    auto load = [&](int base) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + v * kLoad + 4 * threadIdx.x;
            w[v] = i < s1 ? __ldg(reinterpret_cast<const float4*>(weights + i)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    };
    auto make_keys = [&](int base) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = s1 - base - v * kLoad - 4 * static_cast<int>(threadIdx.x);
            keys[v][0] = n > 0 ? weight_key(w[v].x) : 0u;
            keys[v][1] = n > 1 ? weight_key(w[v].y) : 0u;
            keys[v][2] = n > 2 ? weight_key(w[v].z) : 0u;
            keys[v][3] = n > 3 ? weight_key(w[v].w) : 0u;
        }
    };
    // f(key) for each of this thread's weights, and 0 for places without one
    auto visit = [&](auto f) {
        for (int base = s0; base < s1; base += kRound) {
            if (!ONE) {
                load(base);
                make_keys(base);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int c = 0; c < 4; ++c) f(keys[v][c]);
            }
            if (ONE) break;
        }
    };
    if (ONE && choose) load(s0);

    // what needs no selection
    for (int i = kept + part; i < p.out_weight_stride; i += parts) out_w[i] = 0.0f;  // (the copy writes the others)
    for (int i = kept + part; i < p.keep; i += parts) list[i] = -1;
    if (bh % p.num_kv_heads == 0 && part == 0) p.out_lens[b] = kept;
    if (all) {
        for (int i = part; i < len; i += parts) list[i] = i;
        return;
    }
    for (int i = part; i < p.recent; i += parts) list[want + i] = old + i;
    if (!choose) return;

    if (n_cta > 1) cluster_sync();  // every CTA runs, its counts are zero
    else __syncthreads();
    if (ONE) make_keys(s0);
    // The threshold lies among the keys lo + d, 0 <= d <= last; all keys at first.
    uint32_t lo = 1u, last = 0xfffffffeu, share = 0;
    int above = 0;
    // digits of 11, 11 and 10 bits, or in a cluster 11, 8, 8 and 5 (what is
    // sent to every CTA is a histogram at most)
    for (int pass = 0, shift = 32; shift > 0; ++pass) {
        shift -= min(shift, pass == 0 || n_cta == 1 ? 11 : 8);
        visit([&](uint32_t k) {
            const uint32_t d = k - lo;
            if (d <= last) atomicAdd(&hist[d >> shift], 1u);
        });
        __syncthreads();
        const int top = kBins - 1 - kOwnBins * threadIdx.x;  // this thread's bins, largest first
        uint32_t* from = hist;
        if (n_cta > 1) {
            from = sums[pass & 1];
#pragma unroll
            for (int j = 0; j < kOwnBins; ++j) {
                const uint32_t c = hist[top - j];
                if (c != 0) {
                    for (int r = 0; r < n_cta; ++r) red_cluster_add_u32(&from[top - j], r, c);
                    hist[top - j] = 0;
                }
            }
            cluster_sync();
        }
        uint32_t c[kOwnBins], sum = 0;
#pragma unroll
        for (int j = 0; j < kOwnBins; ++j) {
            c[j] = from[top - j];
            from[top - j] = 0;  // (the others add to these sums again after the next step's barrier)
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
            for (int j = 0; j < kOwnBins; ++j) {
                if (before < need && need <= before + c[j]) {
                    pick[0] = top - j;
                    pick[1] = above + before;
                    pick[2] = c[j];
                }
                before += c[j];
            }
        }
        __syncthreads();
        lo += pick[0] << shift;
        last = min((1u << shift) - 1u, 0xffffffffu - lo);  // (the last digit of the first step ends a key earlier)
        above = static_cast<int>(pick[1]);
        share = pick[2];
        if (n_cta > 1 && share <= kShare) break;  // the same for the cluster
        __syncthreads();  // pick and wcount are read before the next step writes them
    }
    uint32_t value = lo;      // the threshold
    uint32_t gt = 0, eq = 0;  // rows above and equal to it before the current round
    if (n_cta > 1) {
        const bool sent = share <= kShare;  // (else all bits are known: that many rows equal the threshold)
        const uint32_t top = lo + last;
        uint32_t n_above = 0, n_share = 0;
        visit([&](uint32_t k) {
            n_above += k > top ? 1u : 0u;
            if (k - lo > last) return;
            if (sent) found[rank * kShare + min(atomicAdd(&own[1], 1u), kShare - 1u)] = k;
            else ++n_share;
        });
        n_above = __reduce_add_sync(0xffffffffu, n_above);
        n_share = __reduce_add_sync(0xffffffffu, n_share);
        if (lane == 0) {
            atomicAdd(&own[0], n_above);
            if (n_share != 0) atomicAdd(&own[1], n_share);
        }
        __syncthreads();
        const int who = warp % n_cta, first = warp / n_cta * 32 + lane, step = THREADS / n_cta;  // a warp or more per CTA
        if (sent && who != rank) {
            const int n = static_cast<int>(min(own[1], static_cast<uint32_t>(kShare)));
            for (int i = first; i < n; i += step) st_cluster_u32(&found[rank * kShare + i], who, found[rank * kShare + i]);
        }
        if (threadIdx.x < n_cta) {
            st_cluster_u32(&above_of[rank], threadIdx.x, own[0]);
            st_cluster_u32(&share_of[rank], threadIdx.x, own[1]);
        }
        cluster_sync();  // (the last one: nothing is written to another CTA from here on)
        if (sent) {
            const int n = static_cast<int>(min(share_of[who], static_cast<uint32_t>(kShare)));
            const uint32_t* theirs = found + who * kShare;
            int larger;
            value = lo + nth_largest<THREADS, uint32_t>(
                want - above, static_cast<int>(share), 0u, last,
                [&](auto f) { for (int i = first; i < n; i += step) f(theirs[i] - lo); }, digits, larger);
            above += larger;
            uint32_t g = 0, e = 0;
            if (who < rank) {
                for (int i = first; i < n; i += step) {
                    g += theirs[i] > value ? 1u : 0u;
                    e += theirs[i] == value ? 1u : 0u;
                }
            }
            g = __reduce_add_sync(0xffffffffu, g);
            e = __reduce_add_sync(0xffffffffu, e);
            if (lane == 0 && who < rank) {
                atomicAdd(&before_cta[0], g + (warp < n_cta ? above_of[who] : 0u));
                atomicAdd(&before_cta[1], e);
            }
        } else if (threadIdx.x < rank) {
            atomicAdd(&before_cta[0], above_of[threadIdx.x]);
            atomicAdd(&before_cta[1], share_of[threadIdx.x]);
        }
        __syncthreads();
        gt = before_cta[0];
        eq = before_cta[1];
    }
    const uint32_t ties = static_cast<uint32_t>(want - above);  // rows equal to the threshold that stay, lowest index first

    // ---- the list.  Rows in order: round, then load (v), then warp, then lane, then the lane's four.
    uint32_t* place = sums[0];  // (free by now) [v][thread]: above | equal << 16 before this thread's four in its piece
    static_assert(V * THREADS <= 2 * kBins, "a word per thread and load");
    for (int base = s0; base < s1; base += kRound) {
        if (!ONE) {
            load(base);
            make_keys(base);
        }
        uint32_t is_above = 0, is_equal = 0;  // bit 4 v + c
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                is_above |= keys[v][c] > value ? 1u << (4 * v + c) : 0u;
                is_equal |= keys[v][c] == value ? 1u << (4 * v + c) : 0u;
            }
        }
        // the counts of the loads (128 at most in a piece), eight bits each
        static_assert(V <= 4, "a word of counts");
        uint32_t n[2] = {0u, 0u};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            n[0] |= static_cast<uint32_t>(__popc(is_above >> (4 * v) & 15u)) << (8 * v);
            n[1] |= static_cast<uint32_t>(__popc(is_equal >> (4 * v) & 15u)) << (8 * v);
        }
        uint32_t s[2] = {n[0], n[1]};
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, s[j], off);
                if (lane >= off) s[j] += o;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            place[v * THREADS + threadIdx.x] = ((s[0] - n[0]) >> (8 * v) & 255u) | ((s[1] - n[1]) >> (8 * v) & 255u) << 16;
            if (lane == 31) piece[v * kWarps + warp] = (s[0] >> (8 * v) & 255u) | (s[1] >> (8 * v) & 255u) << 16;
        }
        __syncthreads();
        // exclusive prefix over the pieces (a round holds at most 16,384 rows: no carry between the halves)
        if (warp == 0) {
            constexpr int P = kPieces / 32;
            static_assert(kPieces % 32 == 0 && kRound <= 16384, "whole lanes; counts fit 16 bits");
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
        for (uint32_t todo = is_above | is_equal; todo != 0; todo &= todo - 1) {
            const int bit = __ffs(todo) - 1, v = bit >> 2;
            const uint32_t at0 = place[v * THREADS + threadIdx.x] + piece[v * kWarps + warp];
            const uint32_t below = (1u << bit) - (1u << (4 * v));  // this thread's rows of the same load before it
            const uint32_t e = eq + (at0 >> 16) + __popc(is_equal & below);
            const uint32_t at = gt + (at0 & 0xffffu) + __popc(is_above & below) + min(e, ties);
            if (((is_above >> bit & 1u) != 0 || e < ties) && at < static_cast<uint32_t>(want))
                list[at] = base + v * kLoad + 4 * static_cast<int>(threadIdx.x) + (bit & 3);
        }
        gt += wcount[0] & 0xffffu;
        eq += wcount[0] >> 16;
        if (ONE) break;
        __syncthreads();
    }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;  // destination rows of a CTA

template <int BPT, int NG>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictCopyParams p) {
    __shared__ long long from[kCopyRows], to[kCopyRows];
    const int heads = p.batch * p.num_kv_heads;
    // the tiles that hold only last rows come first, then each head's others
    const int others = (p.keep - p.recent + kCopyRows - 1) / kCopyRows, lasts = p.tiles - others;
    int i = blockIdx.x, tile, bh;
    if (i < heads * lasts) {
        bh = i / lasts;
        tile = others + i - bh * lasts;
    } else {
        i -= heads * lasts;
        bh = i / others;
        tile = i - bh * others;
    }
    const int b = bh / p.num_kv_heads, h = bh - b * p.num_kv_heads;
    const int r0 = tile * kCopyRows;
    // The grid starts once every CTA of the selection has seen the launches
    // before it end.  CTAs whose rows its list does not decide go ahead; the
    // others wait for it, and every one does before it ends, so that who waits
    // for this grid has waited for both.
    const int len = min(max(__ldcg(p.seq_lens + b), 0), p.max_seq_len);
    const int n = min(kCopyRows, min(len, p.keep) - r0);
    const bool all = len <= p.keep;
    const int want = p.keep - p.recent;
    const bool listed = !all && r0 < want && n > 0;
    pdl_launch_dependents();
    if (listed || n <= 0) pdl_wait_primary();
    if (n <= 0) return;
    if (threadIdx.x < n) {
        const int r = r0 + threadIdx.x;
        const int t = all ? r : (r < want ? __ldcg(p.kept + static_cast<long long>(bh) * p.keep + r) : len - p.keep + r);
        from[threadIdx.x] = kv_row(p.src_map, p.num_kv_heads, b, h, t, p.status);
        to[threadIdx.x] = kv_row(p.dst_map, p.num_kv_heads, b, h, r, p.status);
        p.out_weights[static_cast<long long>(bh) * p.out_weight_stride + r] =
            __ldg(p.weights + static_cast<long long>(bh) * p.weight_stride + t);
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
    if (!listed) pdl_wait_primary();
}

template <int V, int THREADS, bool ONE>
cudaError_t launch_select_v(cudaLaunchConfig_t& cfg, const EvictParams& p) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (p.ctas > 1 && (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire))) {
        const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<V, THREADS, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   8 * kShare * static_cast<int>(sizeof(uint32_t)));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    }
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = p.ctas > 1 ? static_cast<size_t>(p.ctas) * kShare * sizeof(uint32_t) : 0;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<V, THREADS, ONE>, p);
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.num_kv_heads * p.ctas);
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
    // a CTA's stretch; short ones (batches) leave room for two CTAs on an SM
    const long long most = ((static_cast<long long>(p.max_seq_len) - p.recent + p.ctas - 1) / p.ctas + 3) / 4 * 4;
    if (most <= kEvStretch / 4) return launch_select_v<2, 512, true>(cfg, p);
    return most <= kEvStretch ? launch_select_v<4, 1024, true>(cfg, p) : launch_select_v<4, 1024, false>(cfg, p);
}

cudaError_t launch_evict_copy(const EvictCopyParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    EvictCopyParams q = p;
    q.tiles = (p.keep + kCopyRows - 1) / kCopyRows;
    const long long ctas = static_cast<long long>(q.tiles) * p.batch * p.num_kv_heads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
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
    return cudaLaunchKernelEx(&cfg, k, q);
}

}  // namespace tq
