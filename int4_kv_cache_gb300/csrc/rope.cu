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
// Bound by bytes: every row is read and written once.  A CTA takes a token of a
// sequence, whose cosines and sines are computed once into shared memory and
// serve every head of q and k; a thread turns 16 elements at a time.  8,192
// tokens of 64 + 8 heads x 128 (302 MB) take 47.7 us, 6.3 TB/s.  (With two to
// sixteen tokens a CTA, whose output rows are neighbours, or two to six units a
// thread in flight, it took 51 to 74 us; without streaming stores 56 us.)
#include <cuda_fp16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;  // of a row of 256

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
    __shared__ __align__(16) float table[2 * kRopeMaxPairs];  // cosines, then sines
    const int half = p.rotary_dim / 2;
    const int b = blockIdx.y, t = blockIdx.x;
    pdl_wait_primary();
    pdl_launch_dependents();
    for (int j = threadIdx.x; j < half; j += blockDim.x) {
        int axis = 0;
#pragma unroll
        for (int a = 1; a < kRopeAxes; ++a) axis += j >= p.section_end[a - 1] ? 1 : 0;
        const int pos = __ldg(p.positions + (static_cast<long long>(axis) * p.batch + b) * p.n + t);
        const double turns = static_cast<double>(pos) * (static_cast<double>(__ldg(p.inv_freq + j)) * 0.15915494309189535);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
        table[j] = c;
        table[kRopeMaxPairs + j] = p.inverse ? -s : s;
    }
    __syncthreads();
    const int units = p.head_dim / 16, turning = half / 8;
    const int total = (p.q.heads + p.k.heads) * units;
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
        int h = i / units;
        const int u = i - h * units;
        const bool is_k = h >= p.q.heads;
        const RopeRows& rows = is_k ? p.k : p.q;
        if (is_k) h -= p.q.heads;
        const uint16_t* src = rows.x + b * rows.stride_b + t * rows.stride_t + h * rows.stride_h;
        uint16_t* dst = rows.out + ((static_cast<long long>(b) * rows.heads + h) * p.n + t) * p.head_dim;
        const bool turns = u < turning, split = !PAIRS && turns;
        const int e0 = split ? 8 * u : 16 * u, e1 = split ? half + 8 * u : 16 * u + 8;
        uint4 x = __ldcs(reinterpret_cast<const uint4*>(src + e0));
        uint4 y = __ldcs(reinterpret_cast<const uint4*>(src + e1));
        if (turns) {
            const float* c = table + 8 * u;
            if (PAIRS) turn_pairs8(x, y, c, c + kRopeMaxPairs);
            else turn8(x, y, c, c + kRopeMaxPairs);
        }
        __stcs(reinterpret_cast<uint4*>(dst + e0), x);
        __stcs(reinterpret_cast<uint4*>(dst + e1), y);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.n), static_cast<unsigned>(p.batch));
    // as many threads as share a token's units evenly
    const long long total = (static_cast<long long>(p.q.heads) + p.k.heads) * (p.head_dim / 16);
    const long long rounds = (total + kRopeThreads - 1) / kRopeThreads;
    cfg.blockDim = dim3(static_cast<unsigned>(((total + rounds - 1) / rounds + 31) / 32 * 32));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.pairs ? rope_kernel<true> : rope_kernel<false>, p);
}

}  // namespace tq
