// bounds.cu -- per block of cached tokens, kv head and channel: the least and
// the greatest key, which the block selection scores a query against.
//
//     lo_d = min_t k_td,  hi_d = max_t k_td   over the block's rows below stop,
//     k_td = fp16(scale * code + bias)        (one rounding)
//
// A warp takes one block: a lane holds 8 bytes of codes (16 int4 or 8 int8
// elements) of every TOK-th row, turned into packed halves by placing the code
// in the mantissa of 1024 (1024 + n is exact; so is the subtraction) and one
// packed fused multiply-add, so that two channels cost five instructions a
// row.  Rows past stop are replaced by the last row below it, which changes
// neither extreme.  The lanes that share channels meet by shuffles at the end.
// Bound by the cache bytes it reads for a prompt, by latency for a step.
#include <cuda_fp16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kBoundsThreads = 256;

__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i, int bits) {
    // int4: elements (i, i + 4) of the word's eight; int8: (i, i + 2) of its four
    const uint32_t x = bits == 4 ? (w >> (4 * i)) & 0x000F000Fu : (w >> (8 * i)) & 0x00FF00FFu;
    return x | 0x64006400u;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

template <int D, int BITS>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsParams p) {
    constexpr int NG = D / kGroup;
    constexpr int BPT = D * BITS / 8;
    constexpr int LPR = BPT / 8;       // lanes per row
    constexpr int TOK = 32 / LPR;      // rows per pass of the warp
    constexpr int NP = 32 / BITS;      // pairs per lane (two words of NP / 2)
    constexpr int PW = NP / 2;
    static_assert(LPR <= 32, "a row fits one warp");
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const int i = static_cast<int>(item % p.touched);
    const long long bh = item / p.touched;
    if (bh >= static_cast<long long>(p.batch) * p.num_kv_heads) return;
    const int b = static_cast<int>(bh / p.num_kv_heads), h = static_cast<int>(bh - static_cast<long long>(b) * p.num_kv_heads);
    const int start = __ldcg(p.start + b);
    if (start < 0 || start > p.capacity - p.n_rows) {
        if (p.status != nullptr && i == 0 && h == 0 && lane == 0) atomicOr(p.status, TQ_DEV_WRITE_POS);
        return;
    }
    const int stop = start + p.n_rows;
    const int blk = (start >> p.block_shift) + i;
    const int t0 = blk << p.block_shift;
    if (t0 >= stop) return;
    const int rows = min(1 << p.block_shift, stop - t0);
    const long long row0 = kv_row(p.map, p.num_kv_heads, b, h, t0, lane == 0 ? p.status : nullptr);
    const int part = lane % LPR, first = lane / LPR;
    const int g = part * (64 / BITS) / kGroup;
    const uint8_t* codes = p.k_codes + row0 * BPT + part * 8;
    const uint16_t* scale = p.k_scale + row0 * NG + g;
    const uint16_t* bias = p.k_bias + row0 * NG + g;
    __half2 lo[NP], hi[NP];
    const __half2 inf = __float2half2_rn(INFINITY), k1024 = __float2half2_rn(1024.0f);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        lo[j] = inf;
        hi[j] = __hneg2(inf);
    }
    constexpr int U = 8;  // rows of a lane in flight
    for (int r = first; r < rows + first; r += TOK * U) {
        uint2 w[U];
        uint16_t s[U], z[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(r + u * TOK, rows - 1);
            w[u] = __ldcg(reinterpret_cast<const uint2*>(codes + static_cast<long long>(t) * BPT));
            s[u] = __ldg(scale + t * NG);
            z[u] = __ldg(bias + t * NG);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const __half2 s2 = __half2half2(__ushort_as_half(s[u])), z2 = __half2half2(__ushort_as_half(z[u]));
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const __half2 n = __hsub2(as_half2(code_pair(j < PW ? w[u].x : w[u].y, j % PW, BITS)), k1024);
                const __half2 v = __hfma2(n, s2, z2);
                lo[j] = __hmin2(lo[j], v);
                hi[j] = __hmax2(hi[j], v);
            }
        }
    }
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            lo[j] = __hmin2(lo[j], as_half2(__shfl_xor_sync(0xffffffffu, as_u32(lo[j]), off)));
            hi[j] = __hmax2(hi[j], as_half2(__shfl_xor_sync(0xffffffffu, as_u32(hi[j]), off)));
        }
    }
    // one group of lanes writes the least, the next the greatest
    uint16_t* dst = p.bounds + (bh * p.blocks_per_seq + blk) * (2 * D) + part * (64 / BITS);
    auto store = [&](const __half2 (&v)[NP], uint16_t* to) {
        uint32_t out[NP];
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
#pragma unroll
            for (int j = 0; j < PW; j += 2) {  // pairs (j, j + PW) and (j + 1, j + 1 + PW) of the word -> neighbours
                const uint32_t a = as_u32(v[wd * PW + j]), c = as_u32(v[wd * PW + j + 1]);
                out[wd * PW + j / 2] = __byte_perm(a, c, 0x5410);
                out[wd * PW + PW / 2 + j / 2] = __byte_perm(a, c, 0x7632);
            }
        }
#pragma unroll
        for (int j = 0; j < NP; j += 4)
            *reinterpret_cast<uint4*>(to + 2 * j) = make_uint4(out[j], out[j + 1], out[j + 2], out[j + 3]);
    };
    if (TOK == 1 || first == 0) store(lo, dst);
    if (TOK == 1 || first == 1) store(hi, dst + D);
}

}  // namespace

cudaError_t launch_bounds(const BoundsParams& p, cudaStream_t stream) {
    const long long items = static_cast<long long>(p.batch) * p.num_kv_heads * p.touched;
    const long long ctas = (items + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kBoundsThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    using Kern = void (*)(BoundsParams);
    Kern k = nullptr;
    switch (p.head_dim) {
        case 64: k = p.bits == 8 ? bounds_kernel<64, 8> : bounds_kernel<64, 4>; break;
        case 128: k = p.bits == 8 ? bounds_kernel<128, 8> : bounds_kernel<128, 4>; break;
        case 256: k = p.bits == 8 ? bounds_kernel<256, 8> : bounds_kernel<256, 4>; break;
        default: return cudaErrorInvalidValue;
    }
    return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace tq
