// tq_host.h -- host-side pieces of the C-ABI layer shared by its translation
// units: the cache view, argument checks, device facts and the split plan.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_internal.h"

namespace tq {

// A CUDA error as a status (remembered for tq_last_cuda_error()).
tq_status cuda_status(cudaError_t e);

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, unsigned long long na, const void* b, unsigned long long nb) {
    if (na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Tokens of a cache that the operators around the step take (their index
// arithmetic leaves room for blocks, CTAs and pieces behind the last one).
constexpr int32_t kMaxTokens = 1 << 30;

inline bool rotation_flags(uint32_t flags) { return (flags & ~(TQ_ROTATE_K | TQ_ROTATE_V)) == 0; }

inline tq_status check_workspace(const void* ws, size_t have, size_t need) {
    if (ws == nullptr || have < need) return TQ_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ? TQ_ERR_ALIGN : TQ_OK;
}

inline bool supported_dim(int32_t d) { return d == 64 || d == 128 || d == 256; }

// The cache as the kernels see it: the arrays, the sizes, and where each
// logical row lives (tq::RowMap).  A contiguous cache is one page per
// sequence; `capacity` is the logical capacity (max_pages * page_tokens when
// paged).  Field names follow tq_kv_cache so the code below reads the same
// for both layouts.
struct Store {
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint16_t* k_scale;
    uint16_t* k_bias;
    uint16_t* v_scale;
    uint16_t* v_bias;
    int32_t batch, num_kv_heads, head_dim, group_size, capacity, bits;
    tq::RowMap map;
    bool paged;
};

// Pages hold whole pipeline tiles (128 tokens; 64 for head_dim 256), so a
// tile never crosses a page.
constexpr int kPageTokenMultiple = 128;

// The checked view of a cache.
tq_status store_of(const tq_kv_cache* c, Store* st);
tq_status store_of(const tq_paged_kv_cache* c, Store* st);

// The code array of a cache as a 2-D uint8 tensor map for tiles of
// `tile_tokens` tokens (128-byte swizzle).
tq_status make_code_map(CUtensorMap* map, const uint8_t* codes, const Store* c, int tile_tokens);

struct DeviceFacts {
    int sms = 0;
    int mma_ctas[2][3] = {{0, 0, 0}, {0, 0, 0}};  // per code width (4, 8) and head_dim 64 / 128 / 256
    int wide_ctas = 0;  // the one-CTA-per-SM layout (contiguous int4, head_dim 128)
    int simt_ctas[3] = {0, 0, 0};
    // clusters of n CTAs of the cluster-merging kernel held at once, per code
    // width, head_dim, layout (contiguous, paged) and n
    int clusters[2][3][2][tq::kMaxClusterRuns + 1] = {};
    int wide_clusters[tq::kMaxClusterRuns + 1] = {};
};

int dim_index(int d);
tq_status device_facts(DeviceFacts** out);

struct Plan {
    int n_splits, unit_tokens, units;
    bool merged = false;  // the decode merges the runs itself (one run, or one cluster per sequence and kv head)
    int tile_tokens = 0;  // the kernel's pipeline tile
    long long resident = 0;  // CTAs the device holds at once for this kernel
    bool wide = false;    // one 12-warp CTA per SM (else several 4-warp CTAs)
    long long waves = 1;  // ceil(CTAs / resident)
};

inline int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

Plan make_plan(int batch, int hkv, int max_seq_len, int chunk, int tile_tokens, int resident, bool merge,
               const int* cluster_cap = nullptr);
tq_status device_plan(const Store* cache, int max_seq_len, int chunk, tq_impl impl, Plan* pl, bool merge = true);

tq_status check_decode_args(const Store* cache, const uint16_t* q, int32_t hq, const int32_t* seq_lens,
                            int32_t max_seq_len, int32_t chunk, const void* out);
DecodeParams decode_params(const Store* cache, const uint16_t* q, int32_t hq, const int32_t* seq_lens,
                           int32_t max_seq_len, float attn_scale, const Plan& pl, float* pm, float* plv, float* pa,
                           int32_t* status);

}  // namespace tq
