// select.cu -- the blocks of a sequence that a cheap score selects for its
// query ("sparse attention"): for a kv head, a block's score is
//     max over the group's query heads of  sum_d max(q_d lo_d, q_d hi_d),
// an upper bound of q.k over the block's keys (lo, hi: bounds.cu).  The first
// n_first and the last n_last blocks are always listed, the others by score,
// equal scores the lowest index first; the list is ascending.
//
// The sum splits into q+ . hi + q- . lo (q+ = max(q, 0), q- = min(q, 0)), a
// matrix product: mma.sync m16n8k16 with M = 16 blocks, N = the group's heads,
// the bounds going from global memory straight into the A fragments (a lane's
// 16 bytes are two k-steps of one row; the query fragments use the same
// order), so every byte of the bounds is read once, by 16-byte loads.
//
// The list must be that of the exact scores, whatever the order of summation:
// the product's fp32 sums are off by at most kEps * sum |terms|, which a second
// accumulation over absolute values gives.  With eps the largest such bound of
// the row and T the R-th largest fp32 score, the exact R-th largest lies within
// eps of T, so blocks above T + 2 eps are in and those below T - 2 eps are out.
// What lies between (rarely more than one or two blocks) is scored again in
// fp64 (fp16 products are exact there) and ranked by that.
//
// One cluster of CTAs per (sequence, kv head): each CTA scores a stretch of
// blocks and writes the scores into the first CTA's shared memory, which
// selects.  Bound by the bounds' bytes for a batch, by latency for one
// sequence.
#include <cuda_fp16.h>

#include <atomic>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

__device__ __forceinline__ uint32_t ordered_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
    return (u & 0x80000000u) != 0u ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) != 0u ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ uint64_t ordered_key(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return (u >> 63) != 0u ? ~u : (u | 0x8000000000000000ull);
}

// The n-th largest (n >= 1) of the keys visit() hands out, by digits of eight
// bits from the highest in which the keys differ.  `above`: keys larger than
// it.  Every thread calls; visit(f) calls f(key) for this thread's keys.
template <typename K, typename Visit>
__device__ __forceinline__ K nth_largest(int n, Visit visit, uint32_t* hist, int& above) {
    __shared__ K red_lo[kSelWarps], red_hi[kSelWarps];
    __shared__ int pick[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    K lo = ~static_cast<K>(0), hi = 0;
    visit([&](K k) {
        lo = k < lo ? k : lo;
        hi = k > hi ? k : hi;
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const K a = __shfl_xor_sync(0xffffffffu, lo, off), c = __shfl_xor_sync(0xffffffffu, hi, off);
        lo = a < lo ? a : lo;
        hi = c > hi ? c : hi;
    }
    __syncthreads();  // pick and red_* of an earlier call have been read
    if (lane == 0) {
        red_lo[warp] = lo;
        red_hi[warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        lo = red_lo[w] < lo ? red_lo[w] : lo;
        hi = red_hi[w] > hi ? red_hi[w] : hi;
    }
    above = 0;
    const K diff = lo ^ hi;
    int bits = 0;  // the low bits in which keys differ
    for (K d = diff; d != 0; d >>= 1) ++bits;
    const K ones = ~static_cast<K>(0);
    K mask = bits == static_cast<int>(sizeof(K) * 8) ? 0 : ones << bits;  // bits already decided
    K value = hi & mask;
    while (bits > 0) {
        const int take = bits < 8 ? bits : 8, shift = bits - take;
        for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        visit([&](K k) {
            if ((k & mask) == value) atomicAdd(&hist[static_cast<uint32_t>(k >> shift) & ((1u << take) - 1u)], 1u);
        });
        __syncthreads();
        if (warp == 0) {  // lane l holds bins 255 - 8l .. 248 - 8l: counts from the largest digit down
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = hist[255 - 8 * lane - j];
                sum += c[j];
            }
            uint32_t before = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += o;
            }
            before -= sum;
            const uint32_t want = static_cast<uint32_t>(n - above);
            if (before < want && want <= before + sum) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (before < want && want <= before + c[j]) {
                        pick[0] = 255 - 8 * lane - j;
                        pick[1] = above + static_cast<int>(before);
                    }
                    before += c[j];
                }
            }
        }
        __syncthreads();
        value |= static_cast<K>(pick[0]) << shift;
        above = pick[1];
        bits = shift;
        mask = shift == 0 ? ones : ones << shift;
    }
    return value;
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    constexpr int NJ = D / 32;  // 16-byte pieces of a row per lane
    // Every product of 16 terms starts from zero and is added to the sum in
    // fp32: 16 terms cut at 2^-23 of the largest, and D / 8 additions rounded to
    // 2^-24, together below (16 + D / 16) * 2^-23 of the terms' magnitudes
    // (8 * 2^-23 more for the sums that give those magnitudes).
    constexpr float kEps = static_cast<float>(24 + D / 16) * 0x1p-23f;
    extern __shared__ uint32_t keys[];  // the first CTA's: one per block of the sequence
    __shared__ float warp_abs[8 * kSelWarps];  // the first CTA's: largest sum |terms| of every warp
    __shared__ uint32_t hist[256];
    __shared__ int wsum[2][kSelWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int n_cta = p.ctas, rank = static_cast<int>(blockIdx.x) % n_cta;
    const int bh = static_cast<int>(blockIdx.x) / n_cta;
    const int b = bh / p.num_kv_heads;
    const int G = p.group_q;
    pdl_wait_primary();
    pdl_launch_dependents();
    int len = __ldcg(p.seq_lens + b);
    if (len < 0 || len > p.max_seq_len) {
        if (p.status != nullptr && threadIdx.x == 0 && rank == 0 && bh % p.num_kv_heads == 0)
            atomicOr(p.status, TQ_DEV_SEQ_LEN);
        len = min(max(len, 0), p.max_seq_len);
    }
    const int nb = (len + (1 << p.block_shift) - 1) >> p.block_shift;
    int32_t* list = p.blocks + static_cast<long long>(bh) * p.n_select;
    if (nb <= p.n_select) {  // the whole cluster: every block is listed
        for (int i = rank * kSelThreads + threadIdx.x; i < p.n_select; i += n_cta * kSelThreads) list[i] = i < nb ? i : -1;
        return;
    }
    const int c0 = p.n_first, c1 = nb - p.n_last;  // the blocks that compete
    if (n_cta > 1) cluster_sync();  // the first CTA runs: its shared memory may be written

    // ---- scores
    const uint16_t* bounds = p.bounds + static_cast<long long>(bh) * p.blocks_per_seq * (2 * D);
    {
        uint4 qp[NJ], qn[NJ];  // this lane's dims 32 j + 8 tig .. + 7 of head gid: positive and negative parts
        const bool hv = gid < G;
        const uint16_t* q = p.q + (static_cast<long long>(bh) * G + (hv ? gid : 0)) * D + 8 * tig;
        const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (hv) x = *reinterpret_cast<const uint4*>(q + 32 * j);
            const __half2* h = reinterpret_cast<const __half2*>(&x);
            __half2* hp = reinterpret_cast<__half2*>(&qp[j]);
            __half2* hn = reinterpret_cast<__half2*>(&qn[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hp[i] = __hmax2(h[i], zero);
                hn[i] = __hmin2(h[i], zero);
            }
        }
        const int tiles = (nb + 15) / 16, per = (tiles + n_cta - 1) / n_cta;
        const int end = min((rank + 1) * per, tiles);
        float most = 0.0f;
        for (int tile = rank * per + warp; tile < end; tile += kSelWarps) {
            const int r0 = tile * 16 + gid, r1 = r0 + 8;
            const uint16_t* a0 = bounds + static_cast<long long>(min(r0, nb - 1)) * (2 * D) + 8 * tig;
            const uint16_t* a1 = bounds + static_cast<long long>(min(r1, nb - 1)) * (2 * D) + 8 * tig;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, up[4] = {0.0f, 0.0f, 0.0f, 0.0f}, un[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint4 l0 = __ldcg(reinterpret_cast<const uint4*>(a0 + 32 * j));
                const uint4 l1 = __ldcg(reinterpret_cast<const uint4*>(a1 + 32 * j));
                const uint4 h0 = __ldcg(reinterpret_cast<const uint4*>(a0 + D + 32 * j));
                const uint4 h1 = __ldcg(reinterpret_cast<const uint4*>(a1 + D + 32 * j));
                constexpr uint32_t A = 0x7fff7fffu;
                float f[4][4] = {};
                mma_16816(f[0], h0.x, h1.x, h0.y, h1.y, qp[j].x, qp[j].y);
                mma_16816(f[1], h0.z, h1.z, h0.w, h1.w, qp[j].z, qp[j].w);
                mma_16816(f[2], l0.x, l1.x, l0.y, l1.y, qn[j].x, qn[j].y);
                mma_16816(f[3], l0.z, l1.z, l0.w, l1.w, qn[j].z, qn[j].w);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = __fadd_rn(s[i], __fadd_rn(__fadd_rn(f[0][i], f[1][i]), __fadd_rn(f[2][i], f[3][i])));
                mma_16816(up, h0.x & A, h1.x & A, h0.y & A, h1.y & A, qp[j].x, qp[j].y);
                mma_16816(up, h0.z & A, h1.z & A, h0.w & A, h1.w & A, qp[j].z, qp[j].w);
                mma_16816(un, l0.x & A, l1.x & A, l0.y & A, l1.y & A, qn[j].x, qn[j].y);
                mma_16816(un, l0.z & A, l1.z & A, l0.w & A, l1.w & A, qn[j].z, qn[j].w);
            }
            // columns 2 tig, 2 tig + 1 of rows gid (0, 1) and gid + 8 (2, 3)
            const bool v0 = 2 * tig < G, v1 = 2 * tig + 1 < G;
            float m0 = fmaxf(v0 ? s[0] : -INFINITY, v1 ? s[1] : -INFINITY);
            float m1 = fmaxf(v0 ? s[2] : -INFINITY, v1 ? s[3] : -INFINITY);
            // (blocks that are always listed do not compete: whatever their bounds hold)
            if (r0 >= c0 && r0 < c1) most = fmaxf(most, fmaxf(up[0] - un[0], up[1] - un[1]));
            if (r1 >= c0 && r1 < c1) most = fmaxf(most, fmaxf(up[2] - un[2], up[3] - un[3]));
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, off));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
            }
            if (tig == 0 && r0 < nb) st_cluster_u32(&keys[r0], 0, ordered_key(m0));
            if (tig == 1 && r1 < nb) st_cluster_u32(&keys[r1], 0, ordered_key(m1));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
        if (lane == 0) st_cluster_u32(&warp_abs[rank * kSelWarps + warp], 0, __float_as_uint(most));
    }
    if (n_cta > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) return;

    // ---- selection (the first CTA): R of the competing blocks
    const int R = p.n_select - p.n_first - p.n_last;
    float eps = 0.0f;
    for (int i = 0; i < n_cta * kSelWarps; ++i) eps = fmaxf(eps, warp_abs[i]);
    eps *= 2.0f * kEps;
    constexpr uint32_t kIn = 0xffffffffu, kOut = 0u, kOpen = 1u;  // what keys[] becomes (no finite score's key)
    uint64_t open_at = 0;  // the exact score's key from which open blocks are in ...
    int open_ties = 0;     // ... and how many of those equal to it, lowest index first
    double* exact = p.exact + static_cast<long long>(bh) * p.exact_stride;
    if (R > 0) {
        int above;
        const uint32_t tau = nth_largest<uint32_t>(
            R, [&](auto f) { for (int i = c0 + threadIdx.x; i < c1; i += kSelThreads) f(keys[i]); }, hist, above);
        const float t = ordered_value(tau);
        const float up = t + eps, down = t - eps;
        int n_in = 0, n_open = 0;
        for (int i = c0 + threadIdx.x; i < c1; i += kSelThreads) {
            const float v = ordered_value(keys[i]);
            const uint32_t k = v > up ? kIn : (v < down ? kOut : kOpen);
            keys[i] = k;
            n_in += k == kIn;
            n_open += k == kOpen;
        }
        n_in = __reduce_add_sync(0xffffffffu, n_in);
        n_open = __reduce_add_sync(0xffffffffu, n_open);
        if (lane == 0) {
            wsum[0][warp] = n_in;
            wsum[1][warp] = n_open;
        }
        __syncthreads();
        n_in = n_open = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            n_in += wsum[0][w];
            n_open += wsum[1][w];
        }
        if (n_in + n_open > R) {  // the same for the CTA
            // exact scores of the open blocks, a warp each
            for (int i0 = c0 + warp * 32; i0 < c1; i0 += kSelThreads) {
                const int i = i0 + lane;
                uint32_t todo = __ballot_sync(0xffffffffu, i < c1 && keys[i] == kOpen);
                while (todo != 0) {
                    const int blk = i0 + __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint16_t* row = bounds + static_cast<long long>(blk) * (2 * D);
                    double best = -INFINITY;
                    for (int g = 0; g < G; ++g) {
                        const uint16_t* q = p.q + (static_cast<long long>(bh) * G + g) * D;
                        double sum = 0.0;
                        for (int d = lane; d < D; d += 32) {
                            const float x = __half2float(__ushort_as_half(q[d]));
                            const float y = __half2float(__ushort_as_half(row[x > 0.0f ? D + d : d]));
                            sum = fma(static_cast<double>(x), static_cast<double>(y), sum);
                        }
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                        best = sum > best ? sum : best;
                    }
                    if (lane == 0) exact[blk] = best;
                }
            }
            __syncthreads();
            int over;
            open_at = nth_largest<uint64_t>(
                R - n_in,
                [&](auto f) {
                    for (int i = c0 + threadIdx.x; i < c1; i += kSelThreads)
                        if (keys[i] == kOpen) f(ordered_key(exact[i]));
                },
                hist, over);
            open_ties = R - n_in - over;
        } else {
            open_at = 0;
            open_ties = n_open;
        }
        if (n_in + n_open <= R) {  // all of them
            for (int i = c0 + threadIdx.x; i < c1; i += kSelThreads)
                if (keys[i] == kOpen) keys[i] = kIn;
        }
    }
    __syncthreads();

    // ---- the list, in order: first blocks, the selected, last blocks
    for (int i = threadIdx.x; i < p.n_first; i += kSelThreads) list[i] = i;
    for (int i = threadIdx.x; i < p.n_last; i += kSelThreads) list[p.n_select - p.n_last + i] = c1 + i;
    int listed = 0, ties = 0;
    for (int i0 = c0; i0 < c1 && R > 0; i0 += kSelThreads) {
        const int i = i0 + threadIdx.x;
        bool in = false, tie = false;
        if (i < c1) {
            in = keys[i] == kIn;
            if (keys[i] == kOpen) {
                const uint64_t e = ordered_key(exact[i]);
                in = e > open_at;
                tie = e == open_at;
            }
        }
        const uint32_t before = (1u << lane) - 1u;
        const uint32_t bt = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) wsum[1][warp] = __popc(bt);
        __syncthreads();
        int tie_rank = ties + __popc(bt & before);
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) tie_rank += wsum[1][w];
            ties += wsum[1][w];
        }
        in = in || (tie && tie_rank < open_ties);
        const uint32_t bi = __ballot_sync(0xffffffffu, in);
        if (lane == 0) wsum[0][warp] = __popc(bi);
        __syncthreads();
        int at = listed + __popc(bi & before);
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) at += wsum[0][w];
            listed += wsum[0][w];
        }
        if (in && at < R) list[p.n_first + at] = i;
        __syncthreads();
    }
    // scores that are no numbers may leave places: empty ones
    for (int i = listed + threadIdx.x; i < R; i += kSelThreads) list[p.n_first + i] = -1;
}

template <int D>
cudaError_t launch_select_d(cudaLaunchConfig_t& cfg, const SelectParams& p) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxSelectBlocks * static_cast<int>(sizeof(uint32_t)));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    }
    return cudaLaunchKernelEx(&cfg, select_kernel<D>, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.num_kv_heads * p.ctas);
    cfg.blockDim = dim3(kSelThreads);
    const int nb = (p.max_seq_len + (1 << p.block_shift) - 1) >> p.block_shift;
    cfg.dynamicSmemBytes = static_cast<size_t>(nb) * sizeof(uint32_t);
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
    switch (p.head_dim) {
        case 64: return launch_select_d<64>(cfg, p);
        case 128: return launch_select_d<128>(cfg, p);
        case 256: return launch_select_d<256>(cfg, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tq
