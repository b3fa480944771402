// weights.cu -- phase 2 of the decode that accumulates attention weights: the
// log-sum-exp merge of the runs' partial states into the output, and for every
// cached token of a kv head
//     w_t = decay * w_t + sum over the group's heads of e^{s_t - M} / L,
// from the scores s_t that phase 1 kept (log2 units) and the merged maximum M
// and sum L of each head.
//
// One launch: the first CTAs of the grid merge outputs (a CTA per query head, or
// a warp where there are few parts), the others take a stretch of a kv head's
// tokens each, for one sequence as long as leaves one wave of them; every one of them merges the
// heads' m and l itself (a few hundred numbers from L2, while its first scores
// are on their way) rather than wait for another kernel.  Bound by the
// scores: 4 bytes a head and token, written by phase 1 and read here from L2
// while they fit there.  131,072 tokens of 64 heads (33.5 MB) take 7 us of the
// call's 42.6.
#include <math.h>

#include "tq_device.cuh"
#include "tq_hadamard.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightWarps = kWeightThreads / 32;
constexpr int kWeightTokens = 2 * kWeightThreads;  // of a CTA at a time
constexpr int kBatchTokens = 4 * kWeightTokens;    // of a CTA, for a batch

// The merged maximum (log2 units) and sum of one head's parts, by a warp: the
// first 128 parts (m and l read once, at the same time) in registers.
__device__ __forceinline__ void merge_parts(const float* m, const float* l, int n, float& M, float& L) {
    constexpr int H = 4;
    const int lane = threadIdx.x & 31;
    float mc[H], lc[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int c = lane + 32 * i;
        mc[i] = c < n ? __ldcg(m + c) : -INFINITY;
        lc[i] = c < n ? __ldcg(l + c) : 0.0f;
    }
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < H; ++i)
        if (lc[i] > 0.0f) M = fmaxf(M, mc[i]);
    for (int c = lane + 32 * H; c < n; c += 32)
        if (__ldcg(l + c) > 0.0f) M = fmaxf(M, __ldcg(m + c));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < H; ++i)
        if (lc[i] > 0.0f) L = fmaf(exp2f(mc[i] - M), lc[i], L);
    for (int c = lane + 32 * H; c < n; c += 32) {
        const float x = __ldcg(l + c);
        if (x > 0.0f) L = fmaf(exp2f(__ldcg(m + c) - M), x, L);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
}

// The output rows of this CTA's query heads: one head, its parts shared by the
// eight warps, or (few parts) eight heads, a warp each.
template <int D>
__device__ __forceinline__ void merge_outputs(const WeightsParams& p, int heads) {
    constexpr int V = D / 32;
    __shared__ float acc_s[kWeightWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = p.heads_per_cta > 1;  // a warp has a head to itself
    const long long bh = static_cast<long long>(blockIdx.x) * p.heads_per_cta + (alone ? warp : 0);
    if (bh >= heads) return;  // the whole warp; no barrier is ahead of it (alone), or the whole CTA
    const int n = p.n_parts;
    const float* m = p.part_m + bh * n;
    float M, L;
    merge_parts(m, p.part_l + bh * n, n, M, L);
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.0f;
    const int step = alone ? 1 : kWeightWarps;
#pragma unroll 4
    for (int c = alone ? 0 : warp; c < n; c += step) {
        const float w = __ldcg(p.part_l + bh * n + c) > 0.0f ? exp2f(__ldcg(m + c) - M) : 0.0f;
        const float* src = p.part_acc + (bh * n + c) * D + lane * V;
        float x[V];
        if constexpr (V == 2) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            x[0] = v.x;
            x[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i));
                x[i] = v.x;
                x[i + 1] = v.y;
                x[i + 2] = v.z;
                x[i + 3] = v.w;
            }
        }
        if (w != 0.0f) {
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = fmaf(w, x[i], a[i]);
        }
    }
    if (!alone) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc_s[warp][lane * V + i] = a[i];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWeightWarps; ++w) a[i] += acc_s[w][lane * V + i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = L > 0.0f ? __fdiv_rn(a[i], L) : 0.0f;
    if (p.rotate_out) hadamard_warp<V>(a, lane, p.rot_scale);
#pragma unroll
    for (int i = 0; i < V; ++i) p.out[bh * D + lane * V + i] = __half_as_ushort(__float2half_rn(a[i]));
}

template <int D>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const WeightsParams p) {
    __shared__ float head_m[8], head_r[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int heads = p.batch * p.num_q_heads;
    const int merging = (heads + p.heads_per_cta - 1) / p.heads_per_cta;  // CTAs
    if (static_cast<int>(blockIdx.x) < merging) {
        merge_outputs<D>(p, heads);
        return;
    }
    const int G = p.group_q;
    const int item = static_cast<int>(blockIdx.x) - merging;
    const int bh = item / p.chunks, b = bh / p.num_kv_heads;  // (sequence, kv head)
    const int t0 = (item - bh * p.chunks) * p.chunk_tokens;
    const int len = min(max(__ldcg(p.seq_lens + b), 0), p.max_seq_len);
    if (t0 >= len) return;
    const int t1 = min(t0 + p.chunk_tokens, len);
    constexpr int N = kWeightTokens / kWeightThreads;
    const float* scores = p.scores + static_cast<long long>(bh) * p.max_seq_len * G;
    float* weights = p.weights + static_cast<long long>(bh) * p.weight_stride;
    float x[N][8], old[N];
    auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int t = min(base + j * kWeightThreads + static_cast<int>(threadIdx.x), t1 - 1);
            const float* s = scores + static_cast<long long>(t) * G;
            if (G == 8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + i);
                    x[j][4 * i] = v.x;
                    x[j][4 * i + 1] = v.y;
                    x[j][4 * i + 2] = v.z;
                    x[j][4 * i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int g = 0; g < 8; ++g) x[j][g] = g < G ? __ldcg(s + g) : -INFINITY;
            }
            old[j] = p.decay != 0.0f ? __ldcg(weights + t) : 0.0f;
        }
    };
    load(t0);
    {
        float M = 0.0f, L = 0.0f;
        if (warp < G) {
            const long long ph = static_cast<long long>(bh) * G + warp;
            merge_parts(p.part_m + ph * p.n_parts, p.part_l + ph * p.n_parts, p.n_parts, M, L);
        }
        if (lane == 0) {
            // (a head without a sum, every score -inf, adds nothing: no -inf - -inf)
            head_m[warp] = L > 0.0f ? M : 0.0f;
            head_r[warp] = L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f;
        }
    }
    __syncthreads();
    static_assert(kWeightWarps == 8, "a warp per query head");
    for (int base = t0; base < t1; base += kWeightTokens) {
        float sum[N], before[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            sum[j] = 0.0f;
            before[j] = old[j];
#pragma unroll
            for (int g = 0; g < 8; ++g) sum[j] = fmaf(ex2_approx(x[j][g] - head_m[g]), head_r[g], sum[j]);
        }
        if (base + kWeightTokens < t1) load(base + kWeightTokens);  // while these are written
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int t = base + j * kWeightThreads + threadIdx.x;
            if (t < t1) weights[t] = p.decay != 0.0f ? fmaf(p.decay, before[j], sum[j]) : sum[j];
        }
    }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int head_dim, int sms, cudaStream_t stream) {
    WeightsParams q = p;
    const long long rows = static_cast<long long>(p.batch) * p.num_kv_heads;
    const long long wave = 4LL * sms;  // CTAs at once
    const long long whole = (p.max_seq_len + kWeightTokens - 1LL) / kWeightTokens;  // pieces of a sequence
    const long long each = (whole * rows + wave - 1) / wave;
    // One sequence: one wave of equal stretches.  A batch, whose lengths differ:
    // 2,048 tokens a CTA.  (us a call of 32 / 16 int4 sequences of 8,192 tokens /
    // 32 ragged ones of up to 32,768: 95.0 / 47.6 / 188; with 512 tokens a CTA
    // 100 / 50 / 204, with 4,096 96.6 / 50.7 / 189; with four tokens a thread at
    // a time instead of two 95.6 / 48.4 / 191 at best.)
    q.chunk_tokens = p.batch > 1 ? kBatchTokens : static_cast<int32_t>(each < whole ? each : whole) * kWeightTokens;
    q.chunks = (p.max_seq_len + q.chunk_tokens - 1) / q.chunk_tokens;
    // (few: eight at most; with the 15 parts of one short sequence a warp alone
    // takes 2 us longer than eight)
    q.heads_per_cta = p.n_parts <= 8 ? kWeightWarps : 1;
    const long long ctas = (static_cast<long long>(p.batch) * p.num_q_heads + q.heads_per_cta - 1) / q.heads_per_cta + rows * q.chunks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kWeightThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (head_dim) {
        case 64: return cudaLaunchKernelEx(&cfg, weights_kernel<64>, q);
        case 128: return cudaLaunchKernelEx(&cfg, weights_kernel<128>, q);
        case 256: return cudaLaunchKernelEx(&cfg, weights_kernel<256>, q);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tq
