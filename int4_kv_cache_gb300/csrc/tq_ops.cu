// tq_ops.cu -- the extern "C" entry points around the decode step: rotary
// positions, block bounds and sparse decode, the weight-accumulating decode and
// eviction.  Argument checks and dispatch; no device allocation, no host
// synchronisation.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq_host.h"

using namespace tq;

namespace {

constexpr int32_t kMaxListed = 1 << 24;

int block_shift_of(int32_t block_tokens) { return block_tokens == 32 ? 5 : (block_tokens == 64 ? 6 : (block_tokens == 128 ? 7 : -1)); }

// ------------------------------------------------------------------- bounds --
tq_status block_bounds(const Store& c, int32_t block_tokens, const int32_t* start, int32_t n_rows, uint16_t* bounds,
                       int32_t* status, cudaStream_t stream) {
    if (start == nullptr || bounds == nullptr) return TQ_ERR_NULL;
    const int shift = block_shift_of(block_tokens);
    if (shift < 0) return TQ_ERR_UNSUPPORTED;
    if (!aligned16(bounds) || !aligned4(start)) return TQ_ERR_ALIGN;
    if (n_rows < 0) return TQ_ERR_SHAPE;
    if (c.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (n_rows > c.capacity) return TQ_ERR_CAPACITY;
    if (n_rows == 0) return TQ_OK;
    BoundsParams p{};
    p.k_codes = c.k_codes;
    p.k_scale = c.k_scale;
    p.k_bias = c.k_bias;
    p.bounds = bounds;
    p.start = start;
    p.status = status;
    p.batch = c.batch;
    p.num_kv_heads = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.capacity = c.capacity;
    p.bits = c.bits;
    p.n_rows = n_rows;
    p.block_shift = shift;
    p.blocks_per_seq = ceil_div(c.capacity, block_tokens);
    p.touched = (n_rows + block_tokens - 2) / block_tokens + 1;  // rows that start at a block's last row
    if (p.touched > p.blocks_per_seq) p.touched = p.blocks_per_seq;
    p.map = c.map;
    DeviceFacts* f = nullptr;
    const tq_status s = device_facts(&f);
    if (s != TQ_OK) return s;
    return cuda_status(launch_bounds(p, f->sms, stream));
}

// ---------------------------------------------------------------- selection --
struct SelectArgs {
    const uint16_t* bounds;
    const uint16_t* q;
    int32_t batch, hq, hkv, head_dim, capacity;
    const int32_t* seq_lens;
    int32_t max_seq_len, block_tokens, n_select, n_first, n_last;
    int32_t* blocks;
    int32_t* status;
};

tq_status check_select(const SelectArgs& a) {
    if (a.bounds == nullptr || a.q == nullptr || a.seq_lens == nullptr || a.blocks == nullptr) return TQ_ERR_NULL;
    if (a.batch < 1 || a.hkv < 1 || a.hq < 1 || a.hq % a.hkv != 0 || a.capacity < 1 || a.max_seq_len < 1) return TQ_ERR_SHAPE;
    if (!supported_dim(a.head_dim) || a.hq / a.hkv > 8) return TQ_ERR_UNSUPPORTED;
    if (block_shift_of(a.block_tokens) < 0) return TQ_ERR_UNSUPPORTED;
    if (a.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (a.max_seq_len > a.capacity) return TQ_ERR_CAPACITY;
    if (a.n_select < 1 || a.n_select > kMaxListed || a.n_first < 0 || a.n_last < 0 || a.n_first > a.n_select || a.n_last > a.n_select - a.n_first)
        return TQ_ERR_SHAPE;
    const int nb = ceil_div(a.max_seq_len, a.block_tokens);
    if (nb > kMaxSelectBlocks) return TQ_ERR_UNSUPPORTED;
    if (static_cast<long long>(a.batch) * a.hkv * 8 >= (1LL << 31)) return TQ_ERR_SHAPE;
    if (!aligned16(a.bounds) || !aligned16(a.q) || !aligned4(a.blocks) || !aligned4(a.seq_lens)) return TQ_ERR_ALIGN;
    return TQ_OK;
}

// The workspace of a selection: the exact scores of blocks near the border and
// the rotated query.
size_t select_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_seq_len, int32_t block_tokens) {
    const size_t nb = static_cast<size_t>(ceil_div(max_seq_len, block_tokens));
    return align256(static_cast<size_t>(batch) * hkv * nb * sizeof(uint64_t)) +
           align256(static_cast<size_t>(batch) * hq * head_dim * sizeof(uint16_t));
}

uint16_t* rotated_query(const SelectArgs& a, void* workspace) {
    const size_t nb = static_cast<size_t>(ceil_div(a.max_seq_len, a.block_tokens));
    return reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) +
                                       align256(static_cast<size_t>(a.batch) * a.hkv * nb * sizeof(uint64_t)));
}

tq_status rotate_query(SelectArgs& a, void* workspace, cudaStream_t stream) {
    uint16_t* to = rotated_query(a, workspace);
    const tq_status s = cuda_status(launch_rotate_rows(a.q, static_cast<long long>(a.batch) * a.hq, a.head_dim, to,
                                                       rotation_scale(a.head_dim), stream));
    a.q = to;
    return s;
}

tq_status run_select(const SelectArgs& a, void* workspace, cudaStream_t stream) {
    SelectParams p{};
    p.bounds = a.bounds;
    p.q = a.q;
    p.seq_lens = a.seq_lens;
    p.blocks = a.blocks;
    p.exact = static_cast<uint64_t*>(workspace);
    p.status = a.status;
    p.batch = a.batch;
    p.num_kv_heads = a.hkv;
    p.group_q = a.hq / a.hkv;
    p.head_dim = a.head_dim;
    p.max_seq_len = a.max_seq_len;
    p.block_shift = block_shift_of(a.block_tokens);
    p.blocks_per_seq = ceil_div(a.capacity, a.block_tokens);
    p.exact_stride = ceil_div(a.max_seq_len, a.block_tokens);
    p.n_select = a.n_select;
    p.n_first = a.n_first;
    p.n_last = a.n_last;
    // Rows that leave SMs free take CTAs of sixteen warps (eight at head_dim
    // 256, whose tiles are larger), as many (up to eight) as give every warp a
    // tile of 16 blocks while no SM has two; more rows take one CTA of eight
    // warps each, two of which run on an SM.
    DeviceFacts* f = nullptr;
    const tq_status s = device_facts(&f);
    if (s != TQ_OK) return s;
    const long long rows = static_cast<long long>(a.batch) * a.hkv;
    p.wide = rows <= f->sms ? 1 : 0;
    p.ctas = 1;
    const int each = a.head_dim == 256 ? 128 : 256;
    while (p.ctas < 8 && p.exact_stride > each * p.ctas && 2 * rows * p.ctas <= f->sms) p.ctas *= 2;
    cudaError_t e = launch_select(p, stream);
    if (e != cudaSuccess && p.ctas > 1) {  // a cluster the device refused: nothing was queued
        cudaGetLastError();
        p.ctas = 1;
        e = launch_select(p, stream);
    }
    return cuda_status(e);
}

// ---------------------------------------------------------- listed attention --
tq_status check_blocks(const Store& c, const uint16_t* q, int32_t hq, const int32_t* seq_lens, int32_t max_seq_len,
                       const int32_t* blocks, int32_t n_select, int32_t block_tokens, const uint16_t* out) {
    tq_status s = check_decode_args(&c, q, hq, seq_lens, max_seq_len, TQ_DEFAULT_CHUNK, out);
    if (s != TQ_OK) return s;
    if (blocks == nullptr) return TQ_ERR_NULL;
    if (c.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (block_shift_of(block_tokens) < 0) return TQ_ERR_UNSUPPORTED;
    if (n_select < 1 || n_select > kMaxListed || static_cast<long long>(n_select) * block_tokens >= (1LL << 30)) return TQ_ERR_SHAPE;
    if (!aligned4(blocks) || !aligned4(seq_lens)) return TQ_ERR_ALIGN;
    return TQ_OK;
}

// Phase 1 over the listed blocks and, unless it merged its runs itself, the reduce.
tq_status run_blocks(const Store& c, const uint16_t* q, int32_t hq, const int32_t* seq_lens, int32_t max_seq_len,
                     float attn_scale, const int32_t* blocks, int32_t n_select, int32_t block_tokens, uint32_t flags,
                     bool query_rotated, uint8_t* ws, uint16_t* out, int32_t* status, cudaStream_t stream) {
    DeviceFacts* f = nullptr;
    tq_status s = device_facts(&f);
    if (s != TQ_OK) return s;
    const int di = dim_index(c.head_dim), bi = c.bits == 8 ? 1 : 0;
    const int tile = mma_tile_tokens(c.head_dim, c.bits, false);
    const bool merge = !(flags & TQ_ROTATE_V);
    // (The plan's slots and clusters are those of the decode's paged kernel,
    // whose layout this one has; where they differed the plan would be a slower
    // one, and a cluster too many is refused and handled below.)
    const Plan pl = make_plan(c.batch, c.num_kv_heads, n_select * block_tokens, tile, tile, f->sms * f->mma_ctas[bi][di],
                              merge, f->clusters[bi][di][1]);
    if (pl.n_splits > kMaxReduceParts || c.num_kv_heads > 65535 || c.batch > 65535) return TQ_ERR_SHAPE;
    const size_t parts = static_cast<size_t>(c.batch) * hq * pl.n_splits;
    float* pm = reinterpret_cast<float*>(ws);
    float* plv = reinterpret_cast<float*>(ws + align256(parts * sizeof(float)));
    float* pa = reinterpret_cast<float*>(ws + 2 * align256(parts * sizeof(float)));
    DecodeParams p = decode_params(&c, q, hq, seq_lens, max_seq_len, attn_scale, pl, pm, plv, pa, status);
    p.wait_at_start = kWaitAtStart;
    p.rotate_q = (flags & TQ_ROTATE_K) != 0 && !query_rotated ? 1 : 0;
    p.blocks = blocks;
    p.n_list = n_select;
    p.block_tokens = block_tokens;
    p.block_shift = block_shift_of(block_tokens);
    if (pl.merged) {
        p.out = out;
        const cudaError_t e = launch_decode_blocks(p, c.head_dim, stream);
        if (e == cudaSuccess || pl.n_splits == 1) return cuda_status(e);
        cudaGetLastError();  // a refused cluster launch: partial states and the reduce
        p.out = nullptr;
    }
    s = cuda_status(launch_decode_blocks(p, c.head_dim, stream));
    if (s != TQ_OK) return s;
    ReduceParams r{};
    r.part_m = pm;
    r.part_l = plv;
    r.part_acc = pa;
    r.out = out;
    r.batch = c.batch;
    r.num_q_heads = hq;
    r.head_dim = c.head_dim;
    r.n_parts = pl.n_splits;
    r.rotate_out = (flags & TQ_ROTATE_V) ? 1 : 0;
    r.rot_scale = rotation_scale(c.head_dim);
    return cuda_status(launch_reduce(r, stream, true));
}

tq_status blocks_decode(const Store& c, const uint16_t* q, int32_t hq, const int32_t* seq_lens, int32_t max_seq_len,
                        float attn_scale, const int32_t* blocks, int32_t n_select, int32_t block_tokens,
                        uint32_t flags, void* workspace, size_t workspace_bytes, uint16_t* out, int32_t* status,
                        cudaStream_t stream) {
    tq_status s = check_blocks(c, q, hq, seq_lens, max_seq_len, blocks, n_select, block_tokens, out);
    if (s != TQ_OK) return s;
    if (!rotation_flags(flags)) return TQ_ERR_UNSUPPORTED;
    s = check_workspace(workspace, workspace_bytes,
                        tq_sparse_workspace_bytes(c.batch, hq, c.num_kv_heads, c.head_dim, max_seq_len, n_select, block_tokens));
    if (s != TQ_OK) return s;
    uint8_t* ws = static_cast<uint8_t*>(workspace) +
                  select_bytes(c.batch, hq, c.num_kv_heads, c.head_dim, max_seq_len, block_tokens);
    return run_blocks(c, q, hq, seq_lens, max_seq_len, attn_scale, blocks, n_select, block_tokens, flags, false, ws, out,
                      status, stream);
}

tq_status sparse_decode(const Store& c, const uint16_t* bounds, const uint16_t* q, int32_t hq, const int32_t* seq_lens,
                        int32_t max_seq_len, float attn_scale, int32_t block_tokens, int32_t n_select, int32_t n_first,
                        int32_t n_last, uint32_t flags, void* workspace, size_t workspace_bytes, int32_t* blocks,
                        uint16_t* out, int32_t* status, cudaStream_t stream) {
    SelectArgs a{bounds, q, c.batch, hq, c.num_kv_heads, c.head_dim, c.capacity, seq_lens, max_seq_len, block_tokens,
                 n_select, n_first, n_last, blocks, status};
    tq_status s = check_select(a);
    if (s == TQ_OK) s = check_blocks(c, q, hq, seq_lens, max_seq_len, blocks, n_select, block_tokens, out);
    if (s != TQ_OK) return s;
    if (!rotation_flags(flags)) return TQ_ERR_UNSUPPORTED;
    s = check_workspace(workspace, workspace_bytes,
                        tq_sparse_workspace_bytes(c.batch, hq, c.num_kv_heads, c.head_dim, max_seq_len, n_select, block_tokens));
    if (s != TQ_OK) return s;
    if (flags & TQ_ROTATE_K) s = rotate_query(a, workspace, stream);
    if (s == TQ_OK) s = run_select(a, workspace, stream);
    if (s != TQ_OK) return s;
    uint8_t* ws = static_cast<uint8_t*>(workspace) +
                  select_bytes(c.batch, hq, c.num_kv_heads, c.head_dim, max_seq_len, block_tokens);
    return run_blocks(c, a.q, hq, seq_lens, max_seq_len, attn_scale, blocks, n_select, block_tokens, flags, true, ws, out,
                      status, stream);
}

// ------------------------------------------------------------------ weights --
size_t scores_bytes(int32_t batch, int32_t hq, int32_t max_seq_len) {
    return align256(static_cast<size_t>(batch) * hq * max_seq_len * sizeof(float));
}

tq_status decode_weights(const Store& c, const uint16_t* q, int32_t hq, const int32_t* seq_lens, int32_t max_seq_len,
                         float attn_scale, float decay, float* weights, uint32_t flags, void* workspace,
                         size_t workspace_bytes, uint16_t* out, int32_t* status, cudaStream_t stream) {
    tq_status s = check_decode_args(&c, q, hq, seq_lens, max_seq_len, TQ_DEFAULT_CHUNK, out);
    if (s != TQ_OK) return s;
    if (weights == nullptr) return TQ_ERR_NULL;
    if (c.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (!aligned4(weights) || !aligned4(seq_lens)) return TQ_ERR_ALIGN;
    if (!rotation_flags(flags)) return TQ_ERR_UNSUPPORTED;
    if (decay != decay) return TQ_ERR_SHAPE;
    s = check_workspace(workspace, workspace_bytes,
                        tq_weights_workspace_bytes(c.batch, hq, c.num_kv_heads, c.head_dim, max_seq_len));
    if (s != TQ_OK) return s;
    Plan pl;
    s = device_plan(&c, max_seq_len, TQ_DEFAULT_CHUNK, TQ_IMPL_MMA, &pl, false);
    if (s != TQ_OK) return s;
    if (pl.n_splits > kMaxReduceParts || c.num_kv_heads > 65535 || c.batch > 65535) return TQ_ERR_SHAPE;
    const size_t parts = static_cast<size_t>(c.batch) * hq * pl.n_splits;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* scores = reinterpret_cast<float*>(ws);
    ws += scores_bytes(c.batch, hq, max_seq_len);
    float* pm = reinterpret_cast<float*>(ws);
    float* plv = reinterpret_cast<float*>(ws + align256(parts * sizeof(float)));
    float* pa = reinterpret_cast<float*>(ws + 2 * align256(parts * sizeof(float)));
    DecodeParams p = decode_params(&c, q, hq, seq_lens, max_seq_len, attn_scale, pl, pm, plv, pa, status);
    p.wait_at_start = kWaitAtStart;
    p.rotate_q = (flags & TQ_ROTATE_K) ? 1 : 0;
    p.wide = pl.wide ? 1 : 0;
    p.scores = scores;
    CUtensorMap tm_k, tm_v;
    const int tile = mma_tile_tokens(c.head_dim, c.bits, pl.wide);
    s = make_code_map(&tm_k, c.k_codes, &c, tile);
    if (s == TQ_OK) s = make_code_map(&tm_v, c.v_codes, &c, tile);
    if (s != TQ_OK) return s;
    const long long ctas = static_cast<long long>(pl.n_splits) * c.num_kv_heads * c.batch;
    if (c.batch > 1 && ctas > pl.resident) {  // several waves: the longest runs first, as the decode does
        int2* order = reinterpret_cast<int2*>(ws + 2 * align256(parts * sizeof(float)) +
                                              align256(parts * c.head_dim * sizeof(float)));
        OrderParams op{};
        op.seq_lens = seq_lens;
        op.order = order;
        op.status = status;
        op.batch = c.batch;
        op.max_seq_len = max_seq_len;
        op.units = pl.units;
        op.n_splits = pl.n_splits;
        op.unit_tokens = pl.unit_tokens;
        op.tile_tokens = pl.tile_tokens;
        s = cuda_status(launch_order_runs(op, stream));
        if (s != TQ_OK) return s;
        p.order = order;
    }
    s = cuda_status(launch_decode_scores(p, c.head_dim, tm_k, tm_v, stream));
    if (s != TQ_OK) return s;
    WeightsParams w{};
    w.part_m = pm;
    w.part_l = plv;
    w.part_acc = pa;
    w.scores = scores;
    w.seq_lens = seq_lens;
    w.weights = weights;
    w.out = out;
    w.batch = c.batch;
    w.num_q_heads = hq;
    w.num_kv_heads = c.num_kv_heads;
    w.group_q = hq / c.num_kv_heads;
    w.max_seq_len = max_seq_len;
    w.weight_stride = c.capacity;
    w.n_parts = pl.n_splits;
    w.decay = decay;
    w.rotate_out = (flags & TQ_ROTATE_V) ? 1 : 0;
    w.rot_scale = rotation_scale(c.head_dim);
    DeviceFacts* f = nullptr;
    s = device_facts(&f);
    if (s != TQ_OK) return s;
    return cuda_status(launch_weights(w, c.head_dim, f->sms, stream));
}

// ----------------------------------------------------------------- eviction --
tq_status evict(const Store& src, const Store& dst, const float* weights, const int32_t* seq_lens, int32_t max_seq_len,
                int32_t keep, int32_t recent, float* dst_weights, int32_t* dst_lens, int32_t* kept, int32_t* status,
                cudaStream_t stream) {
    if (weights == nullptr || seq_lens == nullptr || dst_weights == nullptr || dst_lens == nullptr || kept == nullptr)
        return TQ_ERR_NULL;
    if (src.batch != dst.batch || src.num_kv_heads != dst.num_kv_heads || src.head_dim != dst.head_dim ||
        src.bits != dst.bits)
        return TQ_ERR_SHAPE;
    if (max_seq_len < 1 || keep < 1 || recent < 0 || recent > keep) return TQ_ERR_SHAPE;
    if (src.capacity > kMaxTokens || dst.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (max_seq_len > src.capacity || keep > dst.capacity) return TQ_ERR_CAPACITY;
    const long long heads = static_cast<long long>(src.batch) * src.num_kv_heads;
    if (heads > 65535) return TQ_ERR_SHAPE;
    if (!aligned16(weights) || !aligned4(seq_lens) || !aligned4(dst_weights) || !aligned4(dst_lens) || !aligned4(kept))
        return TQ_ERR_ALIGN;
    // The rows are read by some CTAs while others write: nothing written may be
    // read, or written twice.  (Rows of one pool are told apart by their pages.)
    struct Range {
        const void* at;
        unsigned long long bytes;
    };
    auto arrays = [](const Store& c, Range* r) {
        const unsigned long long rows = static_cast<unsigned long long>(c.map.num_pages) * c.num_kv_heads * c.map.page_tokens;
        const unsigned long long codes = rows * (c.head_dim * c.bits / 8), sb = rows * (c.head_dim / kGroup * 2);
        const void* at[6] = {c.k_codes, c.v_codes, c.k_scale, c.k_bias, c.v_scale, c.v_bias};
        for (int i = 0; i < 6; ++i) r[i] = {at[i], i < 2 ? codes : sb};
    };
    const unsigned long long lens_bytes = src.batch * 4ull, table_bytes = src.paged ? lens_bytes * src.map.max_pages : 0,
                             dst_table_bytes = dst.paged ? lens_bytes * dst.map.max_pages : 0;
    Range reads[10], writes[9];
    arrays(src, reads);
    arrays(dst, writes);
    reads[6] = {weights, heads * src.capacity * 4ull};
    reads[7] = {seq_lens, lens_bytes};
    reads[8] = {src.map.block_table, table_bytes};
    reads[9] = {dst.map.block_table, dst_table_bytes};
    writes[6] = {dst_weights, heads * dst.capacity * 4ull};
    writes[7] = {dst_lens, lens_bytes};
    writes[8] = {kept, heads * keep * 4ull};
    bool one_pool = src.paged && src.map.page_tokens == dst.map.page_tokens;
    for (int i = 0; i < 6; ++i) one_pool = one_pool && reads[i].at == writes[i].at;
    if (one_pool && src.map.block_table == dst.map.block_table) return TQ_ERR_SHAPE;
    for (int i = 0; i < 9; ++i) {
        for (int j = 0; j < 10; ++j) {
            if (one_pool && i < 6 && j < 6) continue;
            if (overlap(writes[i].at, writes[i].bytes, reads[j].at, reads[j].bytes)) return TQ_ERR_SHAPE;
        }
        for (int j = i + 1; j < 9; ++j)
            if (overlap(writes[i].at, writes[i].bytes, writes[j].at, writes[j].bytes)) return TQ_ERR_SHAPE;
    }
    EvictParams p{};
    p.weights = weights;
    p.seq_lens = seq_lens;
    p.out_weights = dst_weights;
    p.out_lens = dst_lens;
    p.kept = kept;
    p.status = status;
    p.batch = src.batch;
    p.num_kv_heads = src.num_kv_heads;
    p.max_seq_len = max_seq_len;
    p.weight_stride = src.capacity;
    p.out_weight_stride = dst.capacity;
    p.keep = keep;
    p.recent = recent;
    // As many CTAs (up to eight) as hold the weights in registers, and up to
    // eight with 2,048 weights or more each while every SM still has at most
    // one.  (Sixteen, past the portable cluster size, took 31 us where eight
    // took 20 for one sequence of 131,072 tokens: not all clusters ran at once.)
    DeviceFacts* f = nullptr;
    tq_status s = device_facts(&f);
    if (s != TQ_OK) return s;
    p.ctas = 1;
    while (p.ctas < 8 && (max_seq_len > static_cast<long long>(kEvStretch) * p.ctas ||
                          (max_seq_len > 4096 * p.ctas && 2 * heads * p.ctas <= f->sms)))
        p.ctas *= 2;
    cudaError_t e = launch_evict_select(p, stream);
    if (e != cudaSuccess && p.ctas > 1) {  // a cluster the device refused: nothing was queued
        cudaGetLastError();
        p.ctas = 1;
        e = launch_evict_select(p, stream);
    }
    s = cuda_status(e);
    if (s != TQ_OK) return s;
    EvictCopyParams c{};
    c.src_k = src.k_codes;
    c.src_v = src.v_codes;
    c.dst_k = dst.k_codes;
    c.dst_v = dst.v_codes;
    const uint16_t* ssb[4] = {src.k_scale, src.k_bias, src.v_scale, src.v_bias};
    uint16_t* dsb[4] = {dst.k_scale, dst.k_bias, dst.v_scale, dst.v_bias};
    for (int i = 0; i < 4; ++i) {
        c.src_sb[i] = ssb[i];
        c.dst_sb[i] = dsb[i];
    }
    c.kept = kept;
    c.seq_lens = seq_lens;
    c.weights = weights;
    c.out_weights = dst_weights;
    c.weight_stride = src.capacity;
    c.out_weight_stride = dst.capacity;
    c.max_seq_len = max_seq_len;
    c.recent = recent;
    c.status = status;
    c.num_kv_heads = src.num_kv_heads;
    c.batch = src.batch;
    c.head_dim = src.head_dim;
    c.bits = src.bits;
    c.keep = keep;
    c.src_map = src.map;
    c.dst_map = dst.map;
    return cuda_status(launch_evict_copy(c, stream));
}

// --------------------------------------------------------------------- rope --
// Bytes from x to behind the last element of its rows.
unsigned long long rope_extent(const tq_rope_rows* r, int32_t batch, int32_t n, int32_t head_dim) {
    return 2ull * (static_cast<unsigned long long>(batch - 1) * r->stride_b + static_cast<unsigned long long>(n - 1) * r->stride_t +
                   static_cast<unsigned long long>(r->num_heads - 1) * r->stride_h + head_dim);
}

tq_status check_rope_rows(const tq_rope_rows* r) {
    if (r->x == nullptr || r->out == nullptr) return TQ_ERR_NULL;
    if (r->num_heads < 1 || r->num_heads > 65535 || r->stride_b < 0 || r->stride_t < 0 || r->stride_h < 0) return TQ_ERR_SHAPE;
    if (!aligned16(r->x) || !aligned16(r->out) || r->stride_b % 8 != 0 || r->stride_t % 8 != 0 || r->stride_h % 8 != 0)
        return TQ_ERR_ALIGN;
    return TQ_OK;
}

}  // namespace

extern "C" {

tq_status tq_rope_axes(const tq_rope_rows* q, const tq_rope_rows* k, const int32_t* positions, const float* inv_freq,
                       int32_t n_axes, const int32_t* sections, int32_t batch, int32_t n, int32_t head_dim,
                       int32_t rotary_dim, uint32_t flags, void* stream) {
    if (q == nullptr || positions == nullptr || inv_freq == nullptr || sections == nullptr) return TQ_ERR_NULL;
    if (batch < 1 || n < 0 || n_axes < 1) return TQ_ERR_SHAPE;
    if (!supported_dim(head_dim) || n_axes > kRopeAxes || batch > 65535) return TQ_ERR_UNSUPPORTED;
    if ((flags & ~(TQ_ROPE_PAIRS | TQ_ROPE_INVERSE)) != 0) return TQ_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0) return TQ_ERR_SHAPE;
    long long pairs = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (sections[i] < 0) return TQ_ERR_SHAPE;
        pairs += sections[i];
    }
    if (pairs != rotary_dim / 2) return TQ_ERR_SHAPE;
    tq_status s = check_rope_rows(q);
    if (s == TQ_OK && k != nullptr) s = check_rope_rows(k);
    if (s != TQ_OK) return s;
    if (!aligned4(positions) || !aligned4(inv_freq)) return TQ_ERR_ALIGN;
    if (n == 0) return TQ_OK;
    const tq_rope_rows* rows[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        if (rows[i] == nullptr) continue;
        const unsigned long long out_bytes = 2ull * batch * rows[i]->num_heads * n * head_dim;
        for (int j = 0; j < 2; ++j) {
            if (rows[j] == nullptr) continue;
            if (overlap(rows[i]->out, out_bytes, rows[j]->x, rope_extent(rows[j], batch, n, head_dim))) return TQ_ERR_SHAPE;
            if (i != j && overlap(rows[i]->out, out_bytes, rows[j]->out, 2ull * batch * rows[j]->num_heads * n * head_dim))
                return TQ_ERR_SHAPE;
        }
    }
    RopeParams p{};
    p.q = {q->x, q->out, q->stride_b, q->stride_t, q->stride_h, q->num_heads};
    if (k != nullptr) p.k = {k->x, k->out, k->stride_b, k->stride_t, k->stride_h, k->num_heads};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.batch = batch;
    p.n = n;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    int end = 0;
    for (int i = 0; i < kRopeAxes; ++i) {
        if (i < n_axes) end += sections[i];
        p.section_end[i] = end;
    }
    p.pairs = (flags & TQ_ROPE_PAIRS) ? 1 : 0;
    p.inverse = (flags & TQ_ROPE_INVERSE) ? 1 : 0;
    return cuda_status(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

size_t tq_block_bounds_bytes(int32_t batch, int32_t hkv, int32_t head_dim, int32_t capacity, int32_t block_tokens) {
    if (batch < 1 || hkv < 1 || capacity < 1 || !supported_dim(head_dim) || block_shift_of(block_tokens) < 0) return 0;
    return static_cast<size_t>(batch) * hkv * ceil_div(capacity, block_tokens) * head_dim * 2 * sizeof(uint16_t);
}

tq_status tq_kv_block_bounds(const tq_kv_cache* cache, int32_t block_tokens, const int32_t* start, int32_t n_rows,
                             uint16_t* bounds, int32_t* status, void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s : block_bounds(st, block_tokens, start, n_rows, bounds, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_kv_block_bounds(const tq_paged_kv_cache* cache, int32_t block_tokens, const int32_t* start,
                                   int32_t n_rows, uint16_t* bounds, int32_t* status, void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s : block_bounds(st, block_tokens, start, n_rows, bounds, status, static_cast<cudaStream_t>(stream));
}

size_t tq_sparse_workspace_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_seq_len,
                                 int32_t n_select, int32_t block_tokens) {
    if (batch < 1 || hq < 1 || hkv < 1 || !supported_dim(head_dim) || max_seq_len < 1 || n_select < 1 ||
        block_shift_of(block_tokens) < 0 || static_cast<long long>(n_select) * block_tokens >= (1LL << 30))
        return 0;
    return select_bytes(batch, hq, hkv, head_dim, max_seq_len, block_tokens) +
           tq_sdpa_workspace_bytes(batch, hq, hkv, head_dim, n_select * block_tokens, TQ_DEFAULT_CHUNK);
}

tq_status tq_select_blocks(const uint16_t* bounds, const uint16_t* q, int32_t batch, int32_t hq, int32_t hkv,
                           int32_t head_dim, int32_t capacity, const int32_t* seq_lens, int32_t max_seq_len,
                           int32_t block_tokens, int32_t n_select, int32_t n_first, int32_t n_last, uint32_t flags,
                           void* workspace, size_t workspace_bytes, int32_t* blocks, int32_t* status, void* stream) {
    SelectArgs a{bounds, q, batch, hq, hkv, head_dim, capacity, seq_lens, max_seq_len, block_tokens, n_select, n_first,
                 n_last, blocks, status};
    tq_status s = check_select(a);
    if (s != TQ_OK) return s;
    if (!rotation_flags(flags)) return TQ_ERR_UNSUPPORTED;
    s = check_workspace(workspace, workspace_bytes, select_bytes(batch, hq, hkv, head_dim, max_seq_len, block_tokens));
    if (s != TQ_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (flags & TQ_ROTATE_K) s = rotate_query(a, workspace, st);
    return s != TQ_OK ? s : run_select(a, workspace, st);
}

tq_status tq_sdpa_blocks_decode(const tq_kv_cache* cache, const uint16_t* q, int32_t hq, const int32_t* seq_lens,
                                int32_t max_seq_len, float attn_scale, const int32_t* blocks, int32_t n_select,
                                int32_t block_tokens, uint32_t flags, void* workspace, size_t workspace_bytes,
                                uint16_t* out, int32_t* status, void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : blocks_decode(st, q, hq, seq_lens, max_seq_len, attn_scale, blocks, n_select, block_tokens, flags,
                                      workspace, workspace_bytes, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_sdpa_blocks_decode(const tq_paged_kv_cache* cache, const uint16_t* q, int32_t hq,
                                      const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                                      const int32_t* blocks, int32_t n_select, int32_t block_tokens, uint32_t flags,
                                      void* workspace, size_t workspace_bytes, uint16_t* out, int32_t* status,
                                      void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : blocks_decode(st, q, hq, seq_lens, max_seq_len, attn_scale, blocks, n_select, block_tokens, flags,
                                      workspace, workspace_bytes, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_sparse_decode(const tq_kv_cache* cache, const uint16_t* bounds, const uint16_t* q, int32_t hq,
                           const int32_t* seq_lens, int32_t max_seq_len, float attn_scale, int32_t block_tokens,
                           int32_t n_select, int32_t n_first, int32_t n_last, uint32_t flags, void* workspace,
                           size_t workspace_bytes, int32_t* blocks, uint16_t* out, int32_t* status, void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : sparse_decode(st, bounds, q, hq, seq_lens, max_seq_len, attn_scale, block_tokens, n_select,
                                      n_first, n_last, flags, workspace, workspace_bytes, blocks, out, status,
                                      static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_sparse_decode(const tq_paged_kv_cache* cache, const uint16_t* bounds, const uint16_t* q, int32_t hq,
                                 const int32_t* seq_lens, int32_t max_seq_len, float attn_scale, int32_t block_tokens,
                                 int32_t n_select, int32_t n_first, int32_t n_last, uint32_t flags, void* workspace,
                                 size_t workspace_bytes, int32_t* blocks, uint16_t* out, int32_t* status,
                                 void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : sparse_decode(st, bounds, q, hq, seq_lens, max_seq_len, attn_scale, block_tokens, n_select,
                                      n_first, n_last, flags, workspace, workspace_bytes, blocks, out, status,
                                      static_cast<cudaStream_t>(stream));
}

size_t tq_weights_workspace_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_seq_len) {
    const size_t decode = tq_sdpa_workspace_bytes(batch, hq, hkv, head_dim, max_seq_len, TQ_DEFAULT_CHUNK);
    return decode == 0 ? 0 : scores_bytes(batch, hq, max_seq_len) + decode;
}

tq_status tq_sdpa_decode_weights(const tq_kv_cache* cache, const uint16_t* q, int32_t hq, const int32_t* seq_lens,
                                 int32_t max_seq_len, float attn_scale, float decay, float* weights, uint32_t flags,
                                 void* workspace, size_t workspace_bytes, uint16_t* out, int32_t* status,
                                 void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : decode_weights(st, q, hq, seq_lens, max_seq_len, attn_scale, decay, weights, flags, workspace,
                                       workspace_bytes, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_sdpa_decode_weights(const tq_paged_kv_cache* cache, const uint16_t* q, int32_t hq,
                                       const int32_t* seq_lens, int32_t max_seq_len, float attn_scale, float decay,
                                       float* weights, uint32_t flags, void* workspace, size_t workspace_bytes,
                                       uint16_t* out, int32_t* status, void* stream) {
    Store st;
    const tq_status s = store_of(cache, &st);
    return s != TQ_OK ? s
                      : decode_weights(st, q, hq, seq_lens, max_seq_len, attn_scale, decay, weights, flags, workspace,
                                       workspace_bytes, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_kv_evict(const tq_kv_cache* src, const tq_kv_cache* dst, const float* weights, const int32_t* seq_lens,
                      int32_t max_seq_len, int32_t keep, int32_t recent, float* dst_weights, int32_t* dst_lens,
                      int32_t* kept, int32_t* status, void* stream) {
    Store a, c;
    tq_status s = store_of(src, &a);
    if (s == TQ_OK) s = store_of(dst, &c);
    return s != TQ_OK ? s
                      : evict(a, c, weights, seq_lens, max_seq_len, keep, recent, dst_weights, dst_lens, kept, status,
                              static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_kv_evict(const tq_paged_kv_cache* src, const tq_paged_kv_cache* dst, const float* weights,
                            const int32_t* seq_lens, int32_t max_seq_len, int32_t keep, int32_t recent,
                            float* dst_weights, int32_t* dst_lens, int32_t* kept, int32_t* status, void* stream) {
    Store a, c;
    tq_status s = store_of(src, &a);
    if (s == TQ_OK) s = store_of(dst, &c);
    return s != TQ_OK ? s
                      : evict(a, c, weights, seq_lens, max_seq_len, keep, recent, dst_weights, dst_lens, kept, status,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
