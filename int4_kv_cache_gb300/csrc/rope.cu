// rope.cu -- rotary positions with several axes (time, height, width, ...) for
// query and key rows, from the projections' layout into the append's.
//
// Pair i of the rotary_dim / 2 pairs of a row turns by
//     angle = positions[axis(i)][b][t] * inv_freq[i]
// (axis(i): the section that i falls into), fp32 (x1, x2) ->
// (x1 cos - x2 sin, x2 cos + x1 sin), rounded once to fp16.  The angle is
// formed in fp64 and reduced to a fraction of a turn there: positions reach
// 2^31 and an fp32 product would be off by 2^-24 of the angle, whole radians
// far into a sequence.  What is left of the turn is rounded to fp32 (2^-25 of
// half a turn), where sincospif takes over.
//
// Bound by bytes: every row is read and written once.  A CTA takes kTok tokens
// of one sequence; their cosines and sines are computed once into shared
// memory and serve every head of q and k.
#include <cuda_fp16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kRopeThreads = 256;

// A unit: 16 elements that turn together (eight pairs), or 16 plain ones.
__device__ __forceinline__ void turn8(uint4& a, uint4& b, const float* c, const float* s) {
    __half2* x = reinterpret_cast<__half2*>(&a);
    __half2* y = reinterpret_cast<__half2*>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = __half22float2(x[i]), v = __half22float2(y[i]);
        const float2 cc = *reinterpret_cast<const float2*>(c + 2 * i), ss = *reinterpret_cast<const float2*>(s + 2 * i);
        x[i] = __floats2half2_rn(fmaf(u.x, cc.x, -v.x * ss.x), fmaf(u.y, cc.y, -v.y * ss.y));
        y[i] = __floats2half2_rn(fmaf(v.x, cc.x, u.x * ss.x), fmaf(v.y, cc.y, u.y * ss.y));
    }
}

// Eight neighbouring pairs (x0, x1), (x2, x3), ... in two words of four.
__device__ __forceinline__ void turn_pairs8(uint4& a, uint4& b, const float* c, const float* s) {
    __half2* x = reinterpret_cast<__half2*>(&a);
    __half2* y = reinterpret_cast<__half2*>(&b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __half2& h = i < 4 ? x[i] : y[i - 4];
        const float2 u = __half22float2(h);
        h = __floats2half2_rn(fmaf(u.x, c[i], -u.y * s[i]), fmaf(u.y, c[i], u.x * s[i]));
    }
}

template <bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float table[];  // [tokens][2][half]: cosines, sines
    const int half = p.rotary_dim / 2;
    const int b = blockIdx.y;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, p.n - t0);
    pdl_wait_primary();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half, j = i - t * half;
        int axis = 0;
#pragma unroll
        for (int a = 1; a < kRopeAxes; ++a) axis += j >= p.section_end[a - 1] ? 1 : 0;
        const int pos = __ldg(p.positions + (static_cast<long long>(axis) * p.batch + b) * p.n + t0 + t);
        const double turns = static_cast<double>(pos) * (static_cast<double>(__ldg(p.inv_freq + j)) * 0.15915494309189535);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
        table[t * 2 * half + j] = c;
        table[t * 2 * half + half + j] = p.inverse ? -s : s;
    }
    __syncthreads();
    const int units = p.head_dim / 16, turning = half / 8;
    const int heads = p.q.heads + p.k.heads;
    // consecutive threads: the units of a row, then the tokens of a head (whose
    // output rows are neighbours), then the heads
    const int per_head = units * nt, total = heads * per_head;
    constexpr int U = 3;  // units of a thread in flight
    for (int i0 = threadIdx.x; i0 < total; i0 += U * kRopeThreads) {
        uint4 x[U], y[U];
        uint16_t* dst[U];
        int e0[U], e1[U], at[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k * kRopeThreads;
            if (i >= total) break;
            int h = i / per_head;
            const int r = i - h * per_head;
            const int t = r / units, u = r - t * units;
            const bool is_k = h >= p.q.heads;
            const RopeRows& rows = is_k ? p.k : p.q;
            if (is_k) h -= p.q.heads;
            const uint16_t* src = rows.x + b * rows.stride_b + static_cast<long long>(t0 + t) * rows.stride_t + h * rows.stride_h;
            dst[k] = rows.out + ((static_cast<long long>(b) * rows.heads + h) * p.n + t0 + t) * p.head_dim;
            const bool turns = u < turning, split = !PAIRS && turns;
            e0[k] = split ? 8 * u : 16 * u;
            e1[k] = split ? half + 8 * u : 16 * u + 8;
            at[k] = turns ? t * 2 * half + 8 * u : -1;
            x[k] = __ldcs(reinterpret_cast<const uint4*>(src + e0[k]));
            y[k] = __ldcs(reinterpret_cast<const uint4*>(src + e1[k]));
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * kRopeThreads >= total) break;
            if (at[k] >= 0) {
                const float* c = table + at[k];
                if (PAIRS) turn_pairs8(x[k], y[k], c, c + half);
                else turn8(x[k], y[k], c, c + half);
            }
            *reinterpret_cast<uint4*>(dst[k] + e0[k]) = x[k];
            *reinterpret_cast<uint4*>(dst[k] + e1[k]) = y[k];
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.n + p.tokens_per_cta - 1) / p.tokens_per_cta),
                       static_cast<unsigned>(p.batch));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.tokens_per_cta) * p.rotary_dim * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.pairs ? rope_kernel<true> : rope_kernel<false>, p);
}

}  // namespace tq
