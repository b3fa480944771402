// chunk.cu -- attention of several query rows per sequence over the cache: a
// chunk of new tokens in causal order (optionally the last `window` tokens
// only), or every row over the whole sequence.  For row r = (token i, head g) of
// (sequence b, kv head h):
//   out = sum_t p_t V_t / sum_t p_t,  p_t = 2^(c q.K_t - m),  lo_i <= t < hi_i,
// with c = attn_scale log2(e) and m the running maximum.
//
// One warp a row: each lane holds D / 32 channels, a token at a time.
#include "tq_device.cuh"
#include "tq_hadamard.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kThreads = 256;

// The cached keys [lo, hi) that row i of a sequence with ql rows and `len` cached ones sees.
__device__ __forceinline__ void row_span(const ChunkParams& p, int i, int ql, int len, int& lo, int& hi) {
    lo = 0;
    hi = len;
    if (p.full) return;
    const int pos = len - ql + i;
    hi = pos + 1 > 0 ? pos + 1 : 0;
    if (p.window > 0 && pos - p.window + 1 > 0) lo = pos - p.window + 1;
}

// E channels from channel E * lane on of cached row `row`, rounded to fp16.
template <int D, int BITS>
__device__ __forceinline__ void load_row(const uint8_t* codes, const uint16_t* scale, const uint16_t* bias, long long row,
                                         int lane, float (&x)[D / 32]) {
    constexpr int E = D / 32;
    const long long g = row * (D / kGroup) + lane * E / kGroup;
    const float s = __half2float(__ushort_as_half(scale[g])), z = __half2float(__ushort_as_half(bias[g]));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        const int code = BITS == 8 ? codes[row * D + d] : (codes[row * (D / 2) + d / 2] >> ((d & 1) * 4)) & 15;
        x[e] = __half2float(__float2half_rn(fminf(fmaxf(fmaf(s, static_cast<float>(code), z), -65504.f), 65504.f)));
    }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) chunk_kernel(ChunkParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const long long rows = static_cast<long long>(p.n) * p.num_q_heads;
    const int b = static_cast<int>(w / rows);
    if (b >= p.batch) return;
    const int hq = static_cast<int>(w % rows % p.num_q_heads), i = static_cast<int>(w % rows / p.num_q_heads);
    const int h = hq / p.group_q;
    int len = p.seq_lens[b], ql = p.q_lens != nullptr ? p.q_lens[b] : p.n;
    if (len < 0 || len > p.max_seq_len || ql < 0 || ql > p.n) {
        if (p.status != nullptr && lane == 0) atomicOr(p.status, TQ_DEV_SEQ_LEN);
        len = min(max(len, 0), p.max_seq_len);
        ql = min(max(ql, 0), p.n);
    }
    if (i >= ql) return;
    int lo, hi;
    row_span(p, i, ql, len, lo, hi);
    float q[E], acc[E] = {};
    const uint16_t* x = p.q + b * p.stride_b + hq * p.stride_h + i * p.stride_t + lane * E;
    halves_to_floats<E>(x, q);
    if (p.rotate_q) {
        hadamard_warp<E>(q, lane, p.rot_scale);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = __half2float(__float2half_rn(q[e]));
    }
    float m = -INFINITY, l = 0.f;
    for (int t = lo; t < hi; ++t) {
        const long long row = kv_row(p.map, p.num_kv_heads, b, h, t, p.status);
        float k[E], v[E];
        load_row<D, BITS>(p.k_codes, p.k_scale, p.k_bias, row, lane, k);
        load_row<D, BITS>(p.v_codes, p.v_scale, p.v_bias, row, lane, v);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.score_scale_log2;
        const float mn = fmaxf(m, s);
        const float f = m == mn ? 1.f : exp2f(m - mn), w1 = mn == -INFINITY ? 0.f : exp2f(s - mn);
        l = l * f + w1;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w1 * v[e]);
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = l > 0.f ? acc[e] / l : 0.f;
    if (p.rotate_out) hadamard_warp<E>(acc, lane, p.rot_scale);
    uint16_t* o = p.out + ((static_cast<long long>(b) * p.n + i) * p.num_q_heads + hq) * D + lane * E;
    floats_to_halves<E>(acc, o);
}

template <int D>
cudaError_t launch_bits(const ChunkParams& p, cudaStream_t stream) {
    const long long warps = static_cast<long long>(p.batch) * p.n * p.num_q_heads;
    const dim3 grid(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
    if (p.bits == 8)
        chunk_kernel<D, 8><<<grid, kThreads, 0, stream>>>(p);
    else
        chunk_kernel<D, 4><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch_bits<64>(p, stream);
    return head_dim == 128 ? launch_bits<128>(p, stream) : launch_bits<256>(p, stream);
}

}  // namespace tq
