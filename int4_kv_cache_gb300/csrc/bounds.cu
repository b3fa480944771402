// bounds.cu -- per block of cached tokens, kv head and channel: the least and
// the greatest key, which the block selection scores a query against.
//
//     lo_d = min_t k_td,  hi_d = max_t k_td   over the block's rows below stop,
//     k_td = fp16(scale_t * code_td + bias_t)
//
// A warp takes a block, 128 channels of it at most, 32 tokens at a time, copied
// (cp.async, two pieces of 32 tokens ahead and on into its next block) into
// its own shared memory; the grid is as many warps as run at once.  A lane
// reads 8 bytes of codes (16 int4 or 8 int8 elements) of every TOK-th token.  A
// code becomes a packed half in the mantissa of 1024 (1024 + n, or 1024 + 16 n
// for the odd int4 elements, which saves their shift; both are exact, and so is
// taking it off again), the value one packed fused multiply-add, and the
// extremes of two tokens' values and those so far one operation each: 17
// operations for the eight elements of an int4 word.  A block that ends early
// repeats its last row, which changes neither extreme.  The lanes that share
// channels halve them among themselves at the end.  Bound by instructions:
// 131,072 tokens of 8 int4 heads x 128 (84 MB) take 23.5 us, 3.6 TB/s, and 18.7
// million warp instructions, of which those operations are 8.9 and the loads
// from shared memory 1.3; the rest, nearly half, are the copies, each block's
// place and end, and the loops (blocks of 128 tokens 22.6 us, of 32 27.7; int8
// 28.0 for 151 MB, 5.4 TB/s; paged 24.6).  With the cache's last tokens still in
// L2 22.0; there the extremes token by token took 25.9, three pieces ahead 22.1;
// as diag(scale) codes + bias on the tensor cores, with fp32 minima and maxima, 36:
// the extremes of fp32 values are twice as many operations.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kBoundsThreads = 128;
constexpr int kBoundsWarps = kBoundsThreads / 32;
constexpr int kPiece = 32;   // tokens copied at a time
constexpr int kAhead = 2;    // pieces in flight

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
struct BCfg {
    static constexpr int NG = D / kGroup;
    static constexpr int BPT = D * BITS / 8;
    static constexpr int DW = D < 128 ? D : 128;     // channels of a warp
    static constexpr int PARTS = D / DW;
    static constexpr int RB = DW * BITS / 8;         // their code bytes of a row
    static constexpr int SEGS = RB / 16;
    static constexpr int LPR = RB / 8;               // lanes of a row
    static constexpr int TOK = 32 / LPR;             // rows side by side
    static constexpr int PW = 16 / BITS;             // packed pairs of a 32-bit word of codes
    static constexpr int NP = 2 * PW;                // of a lane
    static constexpr int CODE_BYTES = kPiece * RB;
    static constexpr int SB_BYTES = kPiece * NG * 2; // a scale or bias piece
    static constexpr int STAGE_BYTES = CODE_BYTES + 2 * SB_BYTES;
    static constexpr int SMEM_BYTES = kBoundsWarps * (kAhead + 1) * STAGE_BYTES;
};

template <int D, int BITS>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsParams p) {
    using C = BCfg<D, BITS>;
    constexpr int NG = C::NG;
    extern __shared__ __align__(128) uint8_t dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seg = lane % C::LPR, tok = lane / C::LPR;  // this lane's 8 bytes of a row, its rows
    uint8_t* ring = dyn + warp * (kAhead + 1) * C::STAGE_BYTES;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int pieces = (1 << p.block_shift) / kPiece;  // of a block

    // Items: the blocks k of each (sequence b, kv head h) that rows [start,
    // stop) touch, and for wide heads which of their channels.  A warp takes
    // every stride-th, always the same channels; the copies run ahead of the
    // values, and what the values need to know of an item waits in `queue`.
    __shared__ long long queue_out[kBoundsWarps][kAhead + 1];
    __shared__ int queue_rows[kBoundsWarps][kAhead + 1];
    const int stride = gridDim.x * kBoundsWarps / C::PARTS;
    int at = blockIdx.x * kBoundsWarps + warp;
    const int part = at % C::PARTS;
    at /= C::PARTS;
    int k = at % p.touched, h = at / p.touched, b = h / p.num_kv_heads;
    h -= b * p.num_kv_heads;
    const int dk = stride % p.touched, dbh = stride / p.touched;
    const int db = dbh / p.num_kv_heads, dh = dbh - db * p.num_kv_heads;
    int f_at = at, f_piece = 0, f_slot = 0, f_q = 0, q = 0;
    int f_rows = 0;      // the item's rows below stop; 0: nothing to do
    long long f_row = 0; // its first row in the cache
    auto locate = [&]() {
        f_rows = 0;
        long long out = 0;
        if (f_at < p.items) {
            const int start = __ldcg(p.start + b);
            if (start < 0 || start > p.capacity - p.n_rows) {
                if (p.status != nullptr && k == 0 && h == 0 && part == 0 && lane == 0) atomicOr(p.status, TQ_DEV_WRITE_POS);
            } else {
                const int blk = (start >> p.block_shift) + k, t0 = blk << p.block_shift;
                f_rows = max(0, min(1 << p.block_shift, start + p.n_rows - t0));
                if (f_rows > 0) {
                    f_row = kv_row(p.map, p.num_kv_heads, b, h, t0, lane == 0 ? p.status : nullptr);
                    out = ((static_cast<long long>(b) * p.num_kv_heads + h) * p.blocks_per_seq + blk) * (2 * D) + part * C::DW;
                }
            }
        }
        if (lane == 0) {
            queue_out[warp][f_q] = out;
            queue_rows[warp][f_q] = f_rows;
        }
        f_q = f_q == kAhead ? 0 : f_q + 1;
        // the next item's place
        k += dk;
        h += dh;
        b += db;
        if (k >= p.touched) {
            k -= p.touched;
            ++h;
        }
        if (h >= p.num_kv_heads) {
            h -= p.num_kv_heads;
            ++b;
        }
    };
    locate();
    constexpr int kSb = C::SB_BYTES / 16;
    auto fetch = [&]() {
        const int n = f_rows - f_piece * kPiece;  // rows of this piece, the last one repeated
        if (n > 0) {
            uint8_t* st = ring + f_slot * C::STAGE_BYTES + lane * 16;
            const long long row = f_row + f_piece * kPiece;
            const uint8_t* src = p.k_codes + row * C::BPT + part * C::RB;
            if (C::PARTS == 1 && n >= kPiece) {  // consecutive bytes
#pragma unroll
                for (int i = 0; i < C::CODE_BYTES; i += 512) cp_async16(st + i, src + lane * 16 + i);
            } else {
#pragma unroll
                for (int i = 0; i < C::CODE_BYTES; i += 512) {
                    const int t = (i / 16 + lane) / C::SEGS, s = (i / 16 + lane) % C::SEGS;
                    cp_async16(st + i, src + min(t, n - 1) * C::BPT + s * 16);
                }
            }
            if (lane < 2 * kSb && (lane % kSb) * (8 / NG) < n)
                cp_async16(st + C::CODE_BYTES, (lane < kSb ? p.k_scale : p.k_bias) + row * NG + (lane % kSb) * 8);
        }
        cp_async_commit();
        f_slot = f_slot == kAhead ? 0 : f_slot + 1;
        if (++f_piece == pieces) {
            f_piece = 0;
            f_at += stride;
            locate();
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();

    int slot = 0;
    for (; at < p.items; at += stride) {
        __syncwarp();
        const int it_rows = queue_rows[warp][q];
        const long long it_out = queue_out[warp][q];
        q = q == kAhead ? 0 : q + 1;
        // this lane's group of channels, within a row's groups
        const int g = part * (C::DW / kGroup) + seg * (64 / BITS) / kGroup;
        __half2 lo[C::NP], hi[C::NP];
        const __half2 inf = __float2half2_rn(INFINITY);
#pragma unroll
        for (int i = 0; i < C::NP; ++i) {
            lo[i] = inf;
            hi[i] = __hneg2(inf);
        }
        for (int piece = 0; piece < pieces; ++piece) {
            __syncwarp();  // the slot fetched into next has been read by every lane
            fetch();
            cp_async_wait<kAhead>();
            __syncwarp();
            const uint8_t* st = ring + slot * C::STAGE_BYTES;
            slot = slot == kAhead ? 0 : slot + 1;
            const int n = it_rows - piece * kPiece;
            if (n <= 0) continue;  // the same for the warp
            const uint16_t* sc = reinterpret_cast<const uint16_t*>(st + C::CODE_BYTES) + g;
            auto values = [&](auto partial) {
                const uint8_t* codes = st + lane * 8;  // row i TOK + tok, 8 bytes from seg
#pragma unroll
                for (int i = 0; i < kPiece / C::TOK; i += 2) {
                    __half2 s2[2], z2[2];  // two rows at a time: an extreme of three values is one operation
                    uint2 w[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int tk = (i + u) * C::TOK + tok, ts = (decltype(partial)::value ? min(tk, n - 1) : tk) * NG;
                        w[u] = *reinterpret_cast<const uint2*>(codes + (i + u) * 256);
                        s2[u] = __half2half2(__ushort_as_half(sc[ts]));
                        z2[u] = __half2half2(__ushort_as_half(sc[C::SB_BYTES / 2 + ts]));
                    }
#pragma unroll
                    for (int wd = 0; wd < 2; ++wd) {
                        __half2 c0[C::PW], c1[C::PW];
                        code_halves<BITS>(wd ? w[0].y : w[0].x, c0);
                        code_halves<BITS>(wd ? w[1].y : w[1].x, c1);
#pragma unroll
                        for (int j = 0; j < C::PW; ++j) {
                            const __half2 v0 = __hfma2(c0[j], s2[0], z2[0]), v1 = __hfma2(c1[j], s2[1], z2[1]);
                            lo[wd * C::PW + j] = __hmin2(lo[wd * C::PW + j], __hmin2(v0, v1));
                            hi[wd * C::PW + j] = __hmax2(hi[wd * C::PW + j], __hmax2(v0, v1));
                        }
                    }
                }
            };
            if (n >= kPiece) values(std::false_type{});
            else values(std::true_type{});
        }
        if (it_rows == 0) continue;  // the same for the warp
        // The least, and the greatest negated (so that both are minima); the
        // TOK lanes of a segment halve them: first the least from the
        // greatest, then words, then pairs of a word.
        uint32_t v[2 * C::NP];
#pragma unroll
        for (int i = 0; i < C::NP; ++i) {
            v[i] = as_u32(lo[i]);
            v[C::NP + i] = as_u32(__hneg2(hi[i]));
        }
        const bool is_hi = (lane & 16) != 0;
        int first = 0;  // the first pair that stays
#pragma unroll
        for (int off = 16, half = C::NP; off >= C::LPR; off >>= 1, half >>= 1) {
            const bool upper = (lane & off) != 0;
            if (off < 16) first += upper ? half : 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[half + i], off);
                v[i] = as_u32(__hmin2(as_half2(upper ? v[half + i] : v[i]), as_half2(other)));
            }
        }
        constexpr int F = 2 * C::NP / C::TOK;  // pairs that stay
        const uint32_t sign = is_hi ? 0x80008000u : 0u;
        uint16_t* dst = p.bounds + it_out + (is_hi ? D : 0) + seg * (64 / BITS);
        // pairs j and j + 1 of a word hold channels j, j + 1 and those PW behind them
        uint32_t o[F];
#pragma unroll
        for (int i = 0; i < F; i += 2) {
            constexpr int H = F < C::PW ? 1 : C::PW / 2;
            const int wd = i / C::PW, k = i % C::PW / 2;
            o[wd * C::PW + k] = __byte_perm(v[i], v[i + 1], 0x5410) ^ sign;
            o[wd * C::PW + H + k] = __byte_perm(v[i], v[i + 1], 0x7632) ^ sign;
        }
        if constexpr (F == 4) {  // whole words: eight consecutive channels
            *reinterpret_cast<uint4*>(dst + 2 * first) = make_uint4(o[0], o[1], o[2], o[3]);
        } else if constexpr (F == C::PW) {
            *reinterpret_cast<uint2*>(dst + 2 * first) = make_uint2(o[0], o[1]);
        } else {
            static_assert(F == 2 && C::PW == 4, "half a word of int4 codes");
            uint16_t* to = dst + (first & ~3) * 2 + (first & 3);
            *reinterpret_cast<uint32_t*>(to) = o[0];
            *reinterpret_cast<uint32_t*>(to + 4) = o[1];
        }
    }
}

template <int D, int BITS>
cudaError_t launch_bounds_d(cudaLaunchConfig_t& cfg, const BoundsParams& p, int sms) {
    using C = BCfg<D, BITS>;
    static std::atomic<int> per_sm[64];
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (known) n = per_sm[dev].load(std::memory_order_acquire);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(bounds_kernel<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, bounds_kernel<D, BITS>, kBoundsThreads, C::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        if (known) per_sm[dev].store(n, std::memory_order_release);
    }
    const long long items = static_cast<long long>(p.batch) * p.num_kv_heads * p.touched * C::PARTS;
    if (items > 0x7fffffffLL - 1000000) return cudaErrorInvalidConfiguration;
    BoundsParams q = p;
    q.items = static_cast<int32_t>(items / C::PARTS);
    const long long want = (items + kBoundsWarps - 1) / kBoundsWarps, most = static_cast<long long>(sms) * n;
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kBoundsThreads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    return cudaLaunchKernelEx(&cfg, bounds_kernel<D, BITS>, q);
}

}  // namespace

cudaError_t launch_bounds(const BoundsParams& p, int sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (p.head_dim) {
        case 64: return p.bits == 8 ? launch_bounds_d<64, 8>(cfg, p, sms) : launch_bounds_d<64, 4>(cfg, p, sms);
        case 128: return p.bits == 8 ? launch_bounds_d<128, 8>(cfg, p, sms) : launch_bounds_d<128, 4>(cfg, p, sms);
        case 256: return p.bits == 8 ? launch_bounds_d<256, 8>(cfg, p, sms) : launch_bounds_d<256, 4>(cfg, p, sms);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tq
