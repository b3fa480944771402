// bounds.cu -- per block of cached tokens, kv head and channel: the least and
// the greatest key, which the block selection scores a query against.
//
//     lo_d = min_t k_td,  hi_d = max_t k_td   over the block's rows below stop,
//     k_td = fp16(scale * code + bias)        (one rounding)
//
// A warp takes one block.  A row's codes lie in LPR lanes, 8 bytes each (16
// int4 or 8 int8 elements), and each of the warp's TOK = 32 / LPR row groups
// takes block / TOK consecutive rows, so that a lane reads the scales and biases
// of four rows at a time.  A code becomes a packed half in the mantissa of 1024
// (1024 + n, or 1024 + 16 n for the odd int4 elements, which saves their shift;
// both are exact, and so is taking it off again) and the value by one packed
// fused multiply-add.  A block that ends early repeats its last row, which
// changes neither extreme.  The lanes that share channels meet by shuffles.
// Bound by the packed half and integer operations, which run at 64 lanes a
// clock (a word of eight int4 elements takes 21 of them): a prompt of 131,072
// tokens x 8 heads x 128 channels is read (84 MB) at about half the copy rate.
#include <cuda_fp16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kBoundsThreads = 256;

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// The codes of a word as packed halves.  int4: pairs j = 0..3 of elements
// (j, j + 4); int8: pairs j = 0, 1 of elements (j, j + 2).
template <int BITS>
__device__ __forceinline__ void code_halves(uint32_t w, __half2 (&n)[16 / BITS]) {
    const __half2 k1024 = __float2half2_rn(1024.0f);
    if constexpr (BITS == 4) {
        const __half2 k16th = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.0f);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const uint32_t x = j == 0 ? w : w >> 8;
            n[j] = __hsub2(as_half2((x & 0x000F000Fu) | 0x64006400u), k1024);
            n[j + 1] = __hfma2(as_half2((x & 0x00F000F0u) | 0x64006400u), k16th, k64);
        }
    } else {
        n[0] = __hsub2(as_half2((w & 0x00FF00FFu) | 0x64006400u), k1024);
        n[1] = __hsub2(as_half2(((w >> 8) & 0x00FF00FFu) | 0x64006400u), k1024);
    }
}

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
    const __half2 inf = __float2half2_rn(INFINITY);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        lo[j] = inf;
        hi[j] = __hneg2(inf);
    }
    auto take = [&](uint2 w, __half2 s2, __half2 z2) {
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
            __half2 n[PW];
            code_halves<BITS>(wd ? w.y : w.x, n);
#pragma unroll
            for (int j = 0; j < PW; ++j) {
                const __half2 v = __hfma2(n[j], s2, z2);
                lo[wd * PW + j] = __hmin2(lo[wd * PW + j], v);
                hi[wd * PW + j] = __hmax2(hi[wd * PW + j], v);
            }
        }
    };
    constexpr int U = 4;  // rows whose scales one load brings
    const int mine = (1 << p.block_shift) / TOK;  // a multiple of 4
    if (rows == 1 << p.block_shift) {
        struct alignas(NG == 1 ? 8 : 16) Scales {
            uint32_t w[U * NG / 2];
        };
        const uint8_t* c0 = codes + static_cast<long long>(first * mine) * BPT;
        const Scales* s0 = reinterpret_cast<const Scales*>(p.k_scale + (row0 + first * mine) * NG);
        const Scales* z0 = reinterpret_cast<const Scales*>(p.k_bias + (row0 + first * mine) * NG);
        const uint32_t pick = (g & 1) != 0 ? 0x3232u : 0x1010u;  // this lane's group of a pair, twice
#pragma unroll 4
        for (int r = 0; r < mine; r += U) {
            uint2 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = __ldg(reinterpret_cast<const uint2*>(c0 + (r + u) * BPT));
            const Scales s = s0[r / U], z = z0[r / U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t sw, zw;
                if constexpr (NG == 1) {  // the word holds rows u & ~1 and u | 1
                    sw = __byte_perm(s.w[u / 2], 0, (u & 1) != 0 ? 0x3232 : 0x1010);
                    zw = __byte_perm(z.w[u / 2], 0, (u & 1) != 0 ? 0x3232 : 0x1010);
                } else if constexpr (NG == 2) {
                    sw = __byte_perm(s.w[u], 0, pick);
                    zw = __byte_perm(z.w[u], 0, pick);
                } else {
                    sw = __byte_perm((g & 2) != 0 ? s.w[2 * u + 1] : s.w[2 * u], 0, pick);
                    zw = __byte_perm((g & 2) != 0 ? z.w[2 * u + 1] : z.w[2 * u], 0, pick);
                }
                take(w[u], as_half2(sw), as_half2(zw));
            }
        }
    } else {
        for (int r = first; r < rows + first; r += TOK * 2 * U) {
            uint2 w[2 * U];
            uint16_t s[2 * U], z[2 * U];
#pragma unroll
            for (int u = 0; u < 2 * U; ++u) {
                const int t = min(r + u * TOK, rows - 1);
                w[u] = __ldg(reinterpret_cast<const uint2*>(codes + static_cast<long long>(t) * BPT));
                s[u] = __ldg(scale + t * NG);
                z[u] = __ldg(bias + t * NG);
            }
#pragma unroll
            for (int u = 0; u < 2 * U; ++u)
                take(w[u], __half2half2(__ushort_as_half(s[u])), __half2half2(__ushort_as_half(z[u])));
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
