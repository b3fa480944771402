// select.cu -- the blocks of a sequence that a cheap score selects for its
// query ("sparse attention"): for a kv head, a block's score is
//     max over the group's query heads of  sum_d max(q_d lo_d, q_d hi_d),
// an upper bound of q.k over the block's keys (lo, hi: bounds.cu), but for the
// bounds' rounding to the nearest fp16.  The first n_first and the last n_last blocks are always listed, the others by score,
// equal scores the lowest index first; the list is ascending.
//
// The sum splits into q+ . hi + q- . lo (q+ = max(q, 0), q- = min(q, 0)), a
// matrix product: mma.sync m16n8k16 with M = 16 blocks, N = the group's heads.
// Each warp copies its tiles of 16 blocks into shared memory (one bulk copy
// each, every byte of the bounds read once) and takes the A fragments from
// there by 16-byte loads (a lane's 16 bytes are two k-steps of one row; the query
// fragments use the same order).
//
// The list must be that of the exact scores, whatever the order of summation:
// the product's fp32 sums are off by at most kEps * sum |terms|, which a second
// accumulation over absolute values gives.  With eps twice the largest such
// bound of the row and T the R-th largest fp32 score, blocks above T + eps are
// in and those below T - eps are out.  What lies between (rarely more than one
// or two blocks) is summed again in pairs of fp32 numbers, each step with its
// exact error (fp16 products are exact in fp32), 48 bits in all, and ranked by
// that.  (In fp64, whose rate is 1/64 here, the few rows with such blocks took
// 12 us longer than the others; with a general ranking even of a few blocks 6 us
// longer, now 2: a batch's step 44.3 -> 41.2 us.)
//
// One cluster of CTAs per (sequence, kv head): each CTA scores a stretch of
// blocks and writes the scores into the first CTA's shared memory, which
// selects.  Bound by latency: 64 of 2,048 blocks x 8 heads (8.4 MB of bounds)
// take 8.9 us, 32 of up to 512 for each of 32 ragged sequences (35 MB) 12.2 us,
// 8 of them the longest rows' scores.
#include <cuda_fp16.h>

#include <atomic>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_radix.cuh"

namespace tq {

namespace {

__device__ __forceinline__ uint32_t ordered_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
    return (u & 0x80000000u) != 0u ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) != 0u ? (k ^ 0x80000000u) : ~k);
}

// A sum held as hi + lo, lo the rounding errors of hi (Knuth's two-sum).
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ void add(Pair& a, float x, float x_lo) {
    const float s = __fadd_rn(a.hi, x), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(x, t));
    a.lo = __fadd_rn(__fadd_rn(a.lo, x_lo), e);
    a.hi = s;
}
// A key in the order of the sums: hi the sum rounded to fp32, lo the rest (an
// infinite sum has none; its lo is no number).
__device__ __forceinline__ uint64_t ordered_key(const Pair& a) {
    const bool finite = fabsf(a.hi) < INFINITY;
    const float hi = finite ? __fadd_rn(a.hi, a.lo) : a.hi;
    const float lo = finite ? __fsub_rn(a.lo, __fsub_rn(hi, a.hi)) : 0.0f;
    return (static_cast<uint64_t>(ordered_key(hi)) << 32) | ordered_key(lo);
}

// 1-D bulk copy into shared memory, completion counted in bytes on bar.
__device__ __forceinline__ void bulk_fetch(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, D == 256 ? 1 : 512 / THREADS) select_kernel(const SelectParams p) {
    constexpr int WARPS = THREADS / 32;
    constexpr int NJ = D / 32;  // 16-byte pieces of a row per lane
    // Every product of 16 terms starts from zero and is added to the sum in
    // fp32: 16 terms cut at 2^-23 of the largest, and D / 8 additions rounded to
    // 2^-24, together below (16 + D / 16) * 2^-23 of the terms' magnitudes
    // (8 * 2^-23 more for the sums that give those magnitudes).  A factor below
    // 2^-14 counts as 2^-14 there: the terms are aligned by their operands'
    // exponents, which end at that of the smallest normal number.
    constexpr float kEps = static_cast<float>(24 + D / 16) * 0x1p-23f;
    constexpr int kTileBytes = 16 * 4 * D;  // the bounds of 16 blocks
    constexpr uint32_t kLost = 0xffffffffu;  // in place of a sum of magnitudes (which has no sign bit)
    extern __shared__ __align__(128) uint8_t dyn[];
    uint8_t* stage = dyn + (threadIdx.x >> 5) * kTileBytes;              // this warp's tile
    uint32_t* keys = reinterpret_cast<uint32_t*>(dyn + WARPS * kTileBytes);  // the first CTA's: one per block of the sequence
    __shared__ uint64_t bar[WARPS];
    __shared__ __align__(16) uint16_t q_s[8 * D];  // the first CTA's: the group's query heads
    // the first CTA's: every warp's largest sum |terms|, least and greatest key
    __shared__ uint32_t warp_abs[8 * WARPS], warp_lo[8 * WARPS], warp_hi[8 * WARPS];
    __shared__ uint32_t hist[2][256];
    __shared__ int wsum[2][WARPS];
    __shared__ uint64_t red_lo[WARPS], red_hi[WARPS];
    __shared__ int open_s[32];        // few open blocks, and their exact scores
    __shared__ uint64_t exact_s[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int n_cta = p.ctas, rank = static_cast<int>(blockIdx.x) % n_cta;
    const int bh = static_cast<int>(blockIdx.x) / n_cta;
    const int b = bh / p.num_kv_heads;
    const int G = p.group_q;
    // every CTA of the cluster runs once all have arrived: then the first one's
    // shared memory may be written
    if (n_cta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_wait_primary();
    pdl_launch_dependents();
    int len = __ldcg(p.seq_lens + b);
    if (rank == 0) {
        for (int i = threadIdx.x; i < 512; i += THREADS) hist[i >> 8][i & 255] = 0;
    }
    if (lane == 0) mbar_init(&bar[warp], 1);
    fence_mbarrier_init();
    __syncwarp();
    uint4 qraw[NJ];  // this lane's dims 32 j + 8 tig .. + 7 of head gid
    {
        const uint16_t* q = p.q + (static_cast<long long>(bh) * G + (gid < G ? gid : 0)) * D + 8 * tig;
#pragma unroll
        for (int j = 0; j < NJ; ++j) qraw[j] = __ldcg(reinterpret_cast<const uint4*>(q + 32 * j));
    }
    if (rank == 0 && warp == 0 && gid < G) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) *reinterpret_cast<uint4*>(q_s + gid * D + 32 * j + 8 * tig) = qraw[j];
    }
    if (n_cta > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (len < 0 || len > p.max_seq_len) {
        if (p.status != nullptr && threadIdx.x == 0 && rank == 0 && bh % p.num_kv_heads == 0)
            atomicOr(p.status, TQ_DEV_SEQ_LEN);
        len = min(max(len, 0), p.max_seq_len);
    }
    const int nb = (len + (1 << p.block_shift) - 1) >> p.block_shift;
    int32_t* list = p.blocks + static_cast<long long>(bh) * p.n_select;
    if (nb <= p.n_select) {  // the whole cluster: every block is listed
        for (int i = rank * THREADS + threadIdx.x; i < p.n_select; i += n_cta * THREADS) list[i] = i < nb ? i : -1;
        return;
    }
    const int c0 = p.n_first, c1 = nb - p.n_last;  // the blocks that compete

    // ---- scores
    const uint16_t* bounds = p.bounds + static_cast<long long>(bh) * p.blocks_per_seq * (2 * D);
    {
        uint4 qp[NJ], qn[NJ];  // the positive and the negative parts (no head: zeros)
        const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint4 x = gid < G ? qraw[j] : make_uint4(0, 0, 0, 0);
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
        uint32_t q_max = 0u, b_max = 0u;  // largest magnitudes, as pairs of fp16 bit patterns
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t w[4] = {qp[j].x | qn[j].x, qp[j].y | qn[j].y, qp[j].z | qn[j].z, qp[j].w | qn[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) q_max = __vmaxu2(q_max, w[i] & 0x7fff7fffu);
        }
        uint32_t least = 0xffffffffu, greatest = 0u, parity = 0u;
        for (int tile = rank * per + warp; tile < end; tile += WARPS) {
            const int rows = min(16, nb - tile * 16);
            if (lane == 0) {
                const uint32_t bytes = static_cast<uint32_t>(rows) * 4 * D;
                fence_proxy_async_shared();  // the last tile has been read (by the warp: __syncwarp below)
                mbar_arrive_expect_tx(&bar[warp], bytes);
                bulk_fetch(stage, bounds + static_cast<long long>(tile) * 16 * (2 * D), bytes, &bar[warp]);
            }
            const int r0 = tile * 16 + gid, r1 = r0 + 8;
            const uint8_t* a0 = stage + min(gid, rows - 1) * (4 * D) + 16 * tig;
            const uint8_t* a1 = stage + min(gid + 8, rows - 1) * (4 * D) + 16 * tig;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, up[4] = {0.0f, 0.0f, 0.0f, 0.0f}, un[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t m0 = 0u, m1 = 0u;  // largest magnitudes of the two rows
            // (each lane has a time limit of its own: the warp goes on or gives up as one)
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bar[warp], parity))) {
                if (p.status != nullptr && lane == 0) atomicOr(p.status, TQ_DEV_TIMEOUT);
                parity = 2u;  // a tile never arrived: the warp's other blocks have no scores
                break;
            }
            parity ^= 1u;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint4 l0 = *reinterpret_cast<const uint4*>(a0 + 64 * j);
                const uint4 l1 = *reinterpret_cast<const uint4*>(a1 + 64 * j);
                const uint4 h0 = *reinterpret_cast<const uint4*>(a0 + 2 * D + 64 * j);
                const uint4 h1 = *reinterpret_cast<const uint4*>(a1 + 2 * D + 64 * j);
                constexpr uint32_t A = 0x7fff7fffu;  // absolute values
                const uint4 ah0 = make_uint4(h0.x & A, h0.y & A, h0.z & A, h0.w & A), ah1 = make_uint4(h1.x & A, h1.y & A, h1.z & A, h1.w & A);
                const uint4 al0 = make_uint4(l0.x & A, l0.y & A, l0.z & A, l0.w & A), al1 = make_uint4(l1.x & A, l1.y & A, l1.z & A, l1.w & A);
                float f[4][4] = {};
                mma_16816(f[0], h0.x, h1.x, h0.y, h1.y, qp[j].x, qp[j].y);
                mma_16816(f[1], h0.z, h1.z, h0.w, h1.w, qp[j].z, qp[j].w);
                mma_16816(f[2], l0.x, l1.x, l0.y, l1.y, qn[j].x, qn[j].y);
                mma_16816(f[3], l0.z, l1.z, l0.w, l1.w, qn[j].z, qn[j].w);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = __fadd_rn(s[i], __fadd_rn(__fadd_rn(f[0][i], f[1][i]), __fadd_rn(f[2][i], f[3][i])));
                mma_16816(up, ah0.x, ah1.x, ah0.y, ah1.y, qp[j].x, qp[j].y);
                mma_16816(up, ah0.z, ah1.z, ah0.w, ah1.w, qp[j].z, qp[j].w);
                mma_16816(un, al0.x, al1.x, al0.y, al1.y, qn[j].x, qn[j].y);
                mma_16816(un, al0.z, al1.z, al0.w, al1.w, qn[j].z, qn[j].w);
                m0 = __vmaxu2(m0, __vmaxu2(__vmaxu2(ah0.x, ah0.y), __vmaxu2(ah0.z, ah0.w)));
                m0 = __vmaxu2(m0, __vmaxu2(__vmaxu2(al0.x, al0.y), __vmaxu2(al0.z, al0.w)));
                m1 = __vmaxu2(m1, __vmaxu2(__vmaxu2(ah1.x, ah1.y), __vmaxu2(ah1.z, ah1.w)));
                m1 = __vmaxu2(m1, __vmaxu2(__vmaxu2(al1.x, al1.y), __vmaxu2(al1.z, al1.w)));
            }
            // columns 2 tig, 2 tig + 1 of rows gid (0, 1) and gid + 8 (2, 3)
            const bool v0 = 2 * tig < G, v1 = 2 * tig + 1 < G;
            float x0 = fmaxf(v0 ? s[0] : -INFINITY, v1 ? s[1] : -INFINITY);
            float x1 = fmaxf(v0 ? s[2] : -INFINITY, v1 ? s[3] : -INFINITY);
            // (blocks that are always listed do not compete: whatever their bounds hold)
            if (r0 >= c0 && r0 < c1) {
                most = fmaxf(most, fmaxf(up[0] - un[0], up[1] - un[1]));
                b_max = __vmaxu2(b_max, m0);
            }
            if (r1 >= c0 && r1 < c1) {
                most = fmaxf(most, fmaxf(up[2] - un[2], up[3] - un[3]));
                b_max = __vmaxu2(b_max, m1);
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            // lanes tig = 0 pass row r0 on, tig = 1 row r1
            const int r = tig == 0 ? r0 : r1;
            if (tig < 2 && r < nb) {
                const uint32_t k = ordered_key(tig == 0 ? x0 : x1);
                st_cluster_u32(&keys[r], 0, k);
                if (r >= c0 && r < c1) {
                    least = min(least, k);
                    greatest = max(greatest, k);
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
        {   // what factors below 2^-14 add: at most 2 D terms of 2^-14 (max |q| + max |bound| + 2^-14)
            const uint32_t qm = __reduce_max_sync(0xffffffffu, max(q_max & 0xffffu, q_max >> 16));
            const uint32_t bm = __reduce_max_sync(0xffffffffu, max(b_max & 0xffffu, b_max >> 16));
            most += 2.0f * D * 0x1p-14f *
                    (__half2float(__ushort_as_half(static_cast<uint16_t>(qm))) +
                     __half2float(__ushort_as_half(static_cast<uint16_t>(bm))) + 0x1p-14f);
            // an infinite bound (a key above fp16's range), whose zeros times
            // infinity are no numbers in the sums above: every block is open
            if (max(qm, bm) >= 0x7c00u) most = INFINITY;
        }
        least = __reduce_min_sync(0xffffffffu, least);
        greatest = __reduce_max_sync(0xffffffffu, greatest);
        if (lane == 0) {
            st_cluster_u32(&warp_abs[rank * WARPS + warp], 0, parity > 1u ? kLost : __float_as_uint(most));
            st_cluster_u32(&warp_lo[rank * WARPS + warp], 0, least);
            st_cluster_u32(&warp_hi[rank * WARPS + warp], 0, greatest);
        }
    }
    if (n_cta > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) return;

    // ---- selection (the first CTA): R of the competing blocks
    const int R = p.n_select - p.n_first - p.n_last;
    for (int i = threadIdx.x; i < p.n_first; i += THREADS) list[i] = i;
    for (int i = threadIdx.x; i < p.n_last; i += THREADS) list[p.n_select - p.n_last + i] = c1 + i;
    if (R == 0) return;
    float eps = 0.0f;
    uint32_t key_lo = 0xffffffffu, key_hi = 0u;
    bool no_scores = false;
    for (int i = lane; i < n_cta * WARPS; i += 32) {
        no_scores |= warp_abs[i] == kLost;
        eps = fmaxf(eps, __uint_as_float(warp_abs[i]));
        key_lo = min(key_lo, warp_lo[i]);
        key_hi = max(key_hi, warp_hi[i]);
    }
    if (__any_sync(0xffffffffu, no_scores)) {  // the same for the CTA: places without a block instead of unknown ones
        for (int i = threadIdx.x; i < R; i += THREADS) list[p.n_first + i] = -1;
        return;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, off));
    eps *= 2.0f * kEps;
    key_lo = __reduce_min_sync(0xffffffffu, key_lo);
    key_hi = __reduce_max_sync(0xffffffffu, key_hi);
    int above;
    const uint32_t tau = nth_largest<THREADS, uint32_t>(
        R, c1 - c0, key_lo, key_hi, [&](auto f) { for (int i = c0 + threadIdx.x; i < c1; i += THREADS) f(keys[i]); }, hist, above);
    const float up = ordered_value(tau) + eps, down = ordered_value(tau) - eps;
    // each warp a stretch of consecutive blocks [w0, w1): in, or open
    const int span = ((c1 - c0 + WARPS - 1) / WARPS + 31) & ~31;
    const int w0 = min(c0 + warp * span, c1), w1 = min(w0 + span, c1);
    auto is_in = [&](int i) { return ordered_value(keys[i]) > up; };
    auto is_open = [&](int i) {
        const float v = ordered_value(keys[i]);
        return !(v > up) && !(v < down);
    };
    auto count = [&](auto a, auto c) {  // how many blocks of each stretch satisfy a, and how many c
        int na = 0, nc = 0;
        for (int i = w0 + lane; i < w1; i += 32) {
            na += a(i) ? 1 : 0;
            nc += c(i) ? 1 : 0;
        }
        na = __reduce_add_sync(0xffffffffu, na);
        nc = __reduce_add_sync(0xffffffffu, nc);
        if (lane == 0) {
            wsum[0][warp] = na;
            wsum[1][warp] = nc;
        }
    };
    auto totals = [&](int& before_a, int& before_c, int& all_a, int& all_c) {
        before_a = before_c = all_a = all_c = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int na = wsum[0][w], nc = wsum[1][w];
            before_a += w < warp ? na : 0;
            before_c += w < warp ? nc : 0;
            all_a += na;
            all_c += nc;
        }
    };
    // the listed blocks in order: those of a, and of those of c the first `most`
    auto list_them = [&](auto a, auto c, int na, int nc, int most) {
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const bool ia = i < w1 && a(i), ic = i < w1 && c(i);
            const uint32_t ba = __ballot_sync(0xffffffffu, ia), bc = __ballot_sync(0xffffffffu, ic);
            const uint32_t below = (1u << lane) - 1u;
            const int rank_c = nc + __popc(bc & below);
            const int at = na + __popc(ba & below) + min(rank_c, most);
            if ((ia || (ic && rank_c < most)) && at < R) list[p.n_first + at] = i;
            na += __popc(ba);
            nc += __popc(bc);
        }
    };
    int before_in, before_open, n_in, n_open;
    count(is_in, is_open);
    __syncthreads();
    totals(before_in, before_open, n_in, n_open);
    if (n_in + n_open <= R) {  // all of them
        list_them(is_in, is_open, before_in, before_open, n_open);
        // scores that are no numbers may leave places: empty ones
        for (int i = n_in + n_open + threadIdx.x; i < R; i += THREADS) list[p.n_first + i] = -1;
        return;
    }
    // ---- exact scores of the open blocks, a warp each, and their rank
    auto exact_score = [&](int blk) -> uint64_t {
        const uint16_t* row = bounds + static_cast<long long>(blk) * (2 * D);
        float lo[NJ], hi[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            lo[j] = __half2float(__ushort_as_half(__ldcg(row + 32 * j + lane)));
            hi[j] = __half2float(__ushort_as_half(__ldcg(row + D + 32 * j + lane)));
        }
        Pair sum[8];  // of the heads
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            sum[g] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float x = g < G ? __half2float(__ushort_as_half(q_s[g * D + 32 * j + lane])) : 0.0f;
                add(sum[g], x == 0.0f ? 0.0f : __fmul_rn(x, x > 0.0f ? hi[j] : lo[j]), 0.0f);
            }
        }
        // the lanes halve the heads among themselves: lane bits 4, 3, 2 name this lane's
#pragma unroll
        for (int off = 16, half = 4; off >= 4; off >>= 1, half >>= 1) {
            const bool upper = (lane & off) != 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const Pair give = upper ? sum[i] : sum[half + i];
                if (upper) sum[i] = sum[half + i];
                add(sum[i], __shfl_xor_sync(0xffffffffu, give.hi, off), __shfl_xor_sync(0xffffffffu, give.lo, off));
            }
        }
#pragma unroll
        for (int off = 2; off > 0; off >>= 1)
            add(sum[0], __shfl_xor_sync(0xffffffffu, sum[0].hi, off), __shfl_xor_sync(0xffffffffu, sum[0].lo, off));
        uint64_t best = lane >> 2 < G ? ordered_key(sum[0]) : 0;
#pragma unroll
        for (int off = 16; off >= 4; off >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        return best;
    };
    if (n_open <= 32) {  // nearly always: every warp ranks all of them, a lane each
        for (int i0 = w0, at = before_open; i0 < w1; i0 += 32) {
            const bool open = i0 + lane < w1 && is_open(i0 + lane);
            const uint32_t who = __ballot_sync(0xffffffffu, open);
            if (open) open_s[at + __popc(who & ((1u << lane) - 1u))] = i0 + lane;
            at += __popc(who);
        }
        __syncthreads();
        for (int j = warp; j < n_open; j += WARPS) {
            const uint64_t k = exact_score(open_s[j]);
            if (lane == 0) exact_s[j] = k;
        }
        __syncthreads();
        const uint64_t mine = lane < n_open ? exact_s[lane] : 0;
        int ahead = 0;
#pragma unroll 4
        for (int j = 0; j < n_open; ++j) {
            const uint64_t o = exact_s[j];
            ahead += o > mine || (o == mine && j < lane) ? 1 : 0;
        }
        const uint32_t chosen = __ballot_sync(0xffffffffu, lane < n_open && ahead < R - n_in);
        for (int i0 = w0, na = before_in, no = before_open; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const bool in = i < w1 && is_in(i), open = i < w1 && is_open(i);
            const uint32_t bi = __ballot_sync(0xffffffffu, in), bo = __ballot_sync(0xffffffffu, open);
            const uint32_t below = (1u << lane) - 1u;
            const int rank_o = no + __popc(bo & below);  // open blocks before this one
            const int at = na + __popc(bi & below) + __popc(rank_o < 32 ? chosen & ((1u << rank_o) - 1u) : chosen);
            if ((in || (open && (chosen >> (rank_o & 31) & 1u) != 0)) && at < R) list[p.n_first + at] = i;
            na += __popc(bi);
            no += __popc(bo);
        }
        return;
    }
    uint64_t* exact = p.exact + static_cast<long long>(bh) * p.exact_stride;
    uint64_t ex_lo = ~0ull, ex_hi = 0ull;
    for (int i0 = c0 + warp * 32; i0 < c1; i0 += THREADS) {
        uint32_t todo = __ballot_sync(0xffffffffu, i0 + lane < c1 && is_open(i0 + lane));
        while (todo != 0) {
            const int blk = i0 + __ffs(todo) - 1;
            todo &= todo - 1;
            const uint64_t best = exact_score(blk);
            if (lane == 0) exact[blk] = best;
            ex_lo = best < ex_lo ? best : ex_lo;
            ex_hi = best > ex_hi ? best : ex_hi;
        }
    }
    if (lane == 0) {
        red_lo[warp] = ex_lo;
        red_hi[warp] = ex_hi;
    }
    for (int i = threadIdx.x; i < 512; i += THREADS) hist[i >> 8][i & 255] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        ex_lo = red_lo[w] < ex_lo ? red_lo[w] : ex_lo;
        ex_hi = red_hi[w] > ex_hi ? red_hi[w] : ex_hi;
    }
    int over;
    const uint64_t border = nth_largest<THREADS, uint64_t>(
        R - n_in, n_open, ex_lo, ex_hi,
        [&](auto f) {
            for (int i = c0 + threadIdx.x; i < c1; i += THREADS)
                if (is_open(i)) f(exact[i]);
        },
        hist, over);
    auto beats = [&](int i) { return is_in(i) || (is_open(i) && exact[i] > border); };
    auto ties = [&](int i) { return is_open(i) && exact[i] == border; };
    count(beats, ties);
    __syncthreads();
    int before_tie, n_tie;
    totals(before_in, before_tie, n_in, n_tie);
    list_them(beats, ties, before_in, before_tie, R - n_in);
}

template <int D, int THREADS>
cudaError_t launch_select_d(cudaLaunchConfig_t& cfg, const SelectParams& p) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(select_kernel<D, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSelectStageBytes + kMaxSelectBlocks * static_cast<int>(sizeof(uint32_t)));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    }
    static_assert(THREADS / 32 * 64 * D <= kSelectStageBytes, "the warps' tiles");
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes += static_cast<size_t>(THREADS / 32) * 64 * D;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, THREADS>, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.num_kv_heads * p.ctas);
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
        case 64: return p.wide ? launch_select_d<64, 512>(cfg, p) : launch_select_d<64, 256>(cfg, p);
        case 128: return p.wide ? launch_select_d<128, 512>(cfg, p) : launch_select_d<128, 256>(cfg, p);
        case 256: return launch_select_d<256, 256>(cfg, p);  // 16 KB a warp
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tq
