// tq_serve.cu -- the extern "C" entry points for several query rows per sequence
// and for the pages of a pool.  Argument checks and dispatch; no device
// allocation, no host synchronisation.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq_host.h"

using namespace tq;

namespace {

// ---------------------------------------------------------------- overlaps --
struct Span {
    const void* at;
    unsigned long long bytes;
};

// Whether one of the first `writes` spans shares a byte with any other (same: two that may be one array).
bool clash(const Span* s, int n, int writes, int same_a = -1, int same_b = -1, int same_c = -1, int same_d = -1) {
    for (int i = 0; i < writes; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j) continue;
            const bool may = (i == same_a && j == same_b) || (i == same_b && j == same_a) || (i == same_c && j == same_d) || (i == same_d && j == same_c);
            if (may && s[i].at == s[j].at) continue;
            if (overlap(s[i].at, s[i].bytes, s[j].at, s[j].bytes)) return true;
        }
    return false;
}

int arrays_of(const Store& c, Span* s) {
    const unsigned long long rows = static_cast<unsigned long long>(c.map.num_pages) * c.num_kv_heads * c.map.page_tokens;
    const unsigned long long codes = rows * (c.head_dim * c.bits / 8), sb = rows * (c.head_dim / kGroup * 2);
    const void* at[6] = {c.k_codes, c.v_codes, c.k_scale, c.k_bias, c.v_scale, c.v_bias};
    for (int i = 0; i < 6; ++i) s[i] = {at[i], i < 2 ? codes : sb};
    return 6;
}

// ------------------------------------------------------------ several rows --
constexpr long long kMaxChunkRows = 1LL << 28;  // n * num_heads

// Longest wait inside the kernel (a tile of keys takes microseconds).
constexpr uint32_t kChunkLimitUs = 2000000;
constexpr int32_t kAllCopies = 0x7fffffff;

// Most CTAs of a call that splits keys (bounds its workspace independently of the device).
constexpr int kMaxChunkParts = 640;

int chunk_rows(int32_t group, int32_t head_dim, int32_t n) {
    return head_dim != 256 && static_cast<long long>(n) * group > 128 ? 256 : 128;
}

// Rows of partial states at most: every part of a call that splits, or every row's of one of each tile.
size_t chunk_part_rows(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t n, int32_t max_seq_len) {
    const long long per = chunk_rows(hq / hkv, head_dim, n), most = kMaxChunkParts * (head_dim == 256 ? 128LL : 256LL);
    const long long items = static_cast<long long>(batch) * hkv * ((static_cast<long long>(n) * (hq / hkv) + per - 1) / per);
    const long long tiles = ceil_div(max_seq_len, chunk_tile_tokens(head_dim));
    return static_cast<size_t>(items > most / per / tiles ? most : items * tiles * per);
}

size_t part_bytes(size_t rows, int32_t head_dim) { return 2 * align256(rows * sizeof(float)) + align256(rows * head_dim * sizeof(float)); }

// What the CTAs' accumulators are emptied into, where a run can be longer than a chain: a
// place for each whole item and for each part of those that are cut into runs of more than a chain.
size_t chain_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t n, int32_t max_seq_len) {
    const long long chains = ceil_div(max_seq_len, kChunkChainKeys), per = chunk_rows(hq / hkv, head_dim, n);
    if (chains == 1) return 0;
    const long long items = static_cast<long long>(batch) * hkv * ((static_cast<long long>(n) * (hq / hkv) + per - 1) / per);
    const long long cut = items < kMaxChunkParts / chains ? items * chains : kMaxChunkParts;
    return static_cast<size_t>(items + cut) * chunk_chain_floats(head_dim) * sizeof(float);
}

size_t chunk_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t n, int32_t max_seq_len) {
    const size_t parts = part_bytes(chunk_part_rows(batch, hq, hkv, head_dim, n, max_seq_len), head_dim) + chain_bytes(batch, hq, hkv, head_dim, n, max_seq_len);
    const size_t decode = tq_sdpa_workspace_bytes(batch, hq, hkv, head_dim, max_seq_len, TQ_DEFAULT_CHUNK);
    return parts > decode ? parts : decode;
}

// Items with a CTA each, and how many runs the keys of each of the others are cut into.
// Times in tiles: a CTA costs its tiles and some six more (start, first copies, output;
// with four in their place 1,024 tokens of two sequences over 8,192 were cut more than
// pays: 229 us for 210, and 300 of three over 5,000 at head_dim 256: 191 for 179), merging
// a launch and the parts' way through memory.  Either all items are cut, or those that
// are left behind the last full wave of whole ones: 512 items of 508 tiles on 152 SMs
// take 3 whole waves and the rest of their time in an eighth of another one, where a
// fourth whole wave would leave most SMs idle.
constexpr int kCtaTiles = 6;
struct ChunkPlan {
    long long whole;
    int splits;
};

ChunkPlan chunk_plan(long long items, int tiles, int sms) {
    ChunkPlan best{0, 1};
    long long cost = -1;
    for (int full = 0; full < 2; ++full) {
        const long long whole = full ? items / sms * sms : 0, rest = items - whole;
        if (full && (whole == 0 || rest == 0)) continue;
        for (int n = 1; n <= tiles && (n == 1 || rest * n <= kMaxChunkParts); ++n) {
            const long long waves = (rest * n + sms - 1) / sms;
            const long long c = whole / sms * (tiles + kCtaTiles) + waves * ((tiles + n - 1) / n + kCtaTiles) + (n > 1 ? 4 + n / 8 : 0);
            if (cost < 0 || c < cost) {
                cost = c;
                best = {whole, n};
            }
        }
    }
    return best;
}

bool chunk_sizes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t n, int32_t max_seq_len) {
    return batch >= 1 && batch <= 65535 && hkv >= 1 && hkv <= 65535 && hq >= 1 && hq % hkv == 0 && hq / hkv <= 8 && supported_dim(head_dim) &&
           n >= 1 && static_cast<long long>(n) * hq <= kMaxChunkRows && max_seq_len >= 1 && max_seq_len <= kMaxTokens;
}

tq_status check_chunk(const Store& c, const tq_query_rows* q, const int32_t* q_lens, const int32_t* seq_lens, int32_t max_seq_len, int32_t window,
                      uint32_t flags, const void* workspace, size_t workspace_bytes, const uint16_t* out, const int32_t* status) {
    if (q == nullptr || q->x == nullptr || seq_lens == nullptr || out == nullptr) return TQ_ERR_NULL;
    if (q->num_heads < 1 || q->num_heads % c.num_kv_heads != 0 || q->n < 0 || q->stride_b < 0 || q->stride_h < 0 || q->stride_t < 0)
        return TQ_ERR_SHAPE;
    if (max_seq_len < 1 || window < 0) return TQ_ERR_SHAPE;
    if (q->num_heads / c.num_kv_heads > 8 || c.capacity > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (!rotation_flags(flags & ~TQ_CHUNK_FULL) || ((flags & TQ_CHUNK_FULL) && window != 0)) return TQ_ERR_UNSUPPORTED;
    if (c.batch > 65535 || c.num_kv_heads > 65535 || static_cast<long long>(q->n) * q->num_heads > kMaxChunkRows) return TQ_ERR_SHAPE;
    if (max_seq_len > c.capacity) return TQ_ERR_CAPACITY;
    if (!aligned16(q->x) || !aligned16(out) || q->stride_b % 8 != 0 || q->stride_h % 8 != 0 || q->stride_t % 8 != 0 || !aligned4(seq_lens) ||
        !aligned4(q_lens) || !aligned4(status))
        return TQ_ERR_ALIGN;
    if (q->n == 0) return TQ_OK;
    const size_t need = chunk_bytes(c.batch, q->num_heads, c.num_kv_heads, c.head_dim, q->n, max_seq_len);
    const tq_status s = check_workspace(workspace, workspace_bytes, need);
    if (s != TQ_OK) return s;
    const unsigned long long extent = 2ull * (static_cast<unsigned long long>(c.batch - 1) * q->stride_b + static_cast<unsigned long long>(q->n - 1) * q->stride_t +
                                              static_cast<unsigned long long>(q->num_heads - 1) * q->stride_h + c.head_dim);
    // written: out, workspace, status
    Span sp[16] = {{out, 2ull * c.batch * q->n * q->num_heads * c.head_dim}, {workspace, need}, {status, status != nullptr ? 4ull : 0ull}, {q->x, extent},
                   {seq_lens, 4ull * c.batch}, {q_lens, q_lens != nullptr ? 4ull * c.batch : 0ull},
                   {c.map.block_table, c.paged ? 4ull * c.batch * c.map.max_pages : 0ull}};
    const int n = 7 + arrays_of(c, sp + 7);
    return clash(sp, n, 3) ? TQ_ERR_SHAPE : TQ_OK;
}

tq_status chunk(const Store& c, const tq_query_rows* q, const int32_t* q_lens, const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                int32_t window, uint32_t flags, void* workspace, uint16_t* out, int32_t* status, cudaStream_t stream, uint32_t limit_us = kChunkLimitUs,
                int32_t copies = kAllCopies) {
    ChunkParams p{};
    p.limit_us = limit_us;
    p.copies = copies;
    p.q = q->x;
    p.stride_b = q->stride_b;
    p.stride_h = q->stride_h;
    p.stride_t = q->stride_t;
    p.q_lens = q_lens;
    p.seq_lens = seq_lens;
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.k_scale = c.k_scale;
    p.k_bias = c.k_bias;
    p.v_scale = c.v_scale;
    p.v_bias = c.v_bias;
    p.out = out;
    p.status = status;
    p.batch = c.batch;
    p.num_q_heads = q->num_heads;
    p.num_kv_heads = c.num_kv_heads;
    p.group_q = q->num_heads / c.num_kv_heads;
    p.n = q->n;
    p.max_seq_len = max_seq_len;
    p.capacity = c.capacity;
    p.bits = c.bits;
    // (a window past the longest sequence is one of that length, so that positions less a window stay within 32 bits)
    p.window = window = window < max_seq_len ? window : max_seq_len;
    p.full = (flags & TQ_CHUNK_FULL) ? 1 : 0;
    p.rotate_q = (flags & TQ_ROTATE_K) ? 1 : 0;
    p.rotate_out = (flags & TQ_ROTATE_V) ? 1 : 0;
    // (a scale of 0 as one that makes every score vanish: minus infinity stays what it is)
    const float scale = (attn_scale < 0.f ? -attn_scale : attn_scale) * 1.4426950408889634f;
    p.score_scale_log2 = scale > 1e-30f ? scale : 1e-30f;
    p.negate_q = attn_scale < 0.f ? 1 : 0;
    p.rot_scale = rotation_scale(c.head_dim);
    p.map = c.map;
    DeviceFacts* f = nullptr;
    const tq_status s = device_facts(&f);
    if (s != TQ_OK) return s;
    const long long rows = static_cast<long long>(p.n) * p.group_q;
    const int tile = chunk_tile_tokens(c.head_dim);
    p.rows_per_item = chunk_rows(p.group_q, c.head_dim, p.n);
    p.m_items = ceil_div(rows, p.rows_per_item);
    const long long items = static_cast<long long>(c.batch) * c.num_kv_heads * p.m_items;
    // the most keys an item sees: all of them, or a window behind each of its tokens
    long long keys = max_seq_len;
    if (window > 0 && window + static_cast<long long>(p.rows_per_item / p.group_q) + 1 < keys) keys = window + p.rows_per_item / p.group_q + 1;
    if (items >= (1LL << 30)) return TQ_ERR_SHAPE;
    const ChunkPlan pl = chunk_plan(items, ceil_div(keys, tile), f->sms);
    p.n_splits = pl.splits;
    p.whole = pl.splits == 1 ? 0 : static_cast<int32_t>(pl.whole);
    if (p.group_q > 1) {
        const RowMap d = with_page_divisor({nullptr, p.group_q, 0, 0, 0, 0});
        p.group_magic = d.page_magic;
        p.group_shift = d.page_shift;
    }
    const size_t part_rows = chunk_part_rows(c.batch, q->num_heads, c.num_kv_heads, c.head_dim, q->n, max_seq_len);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part_m = reinterpret_cast<float*>(ws);
    p.part_l = reinterpret_cast<float*>(ws + align256(part_rows * sizeof(float)));
    p.part_acc = reinterpret_cast<float*>(ws + 2 * align256(part_rows * sizeof(float)));
    p.chains = reinterpret_cast<float*>(ws + part_bytes(part_rows, c.head_dim));
    return cuda_status(launch_chunk(p, c.head_dim, stream));
}

// One row a sequence, contiguous: what the decode is for (a 128-row tile would hold
// group_q rows; 16 sequences of 16 heads over up to 1,500 tokens: 31 us in tiles).
bool is_decode(const Store& c, const tq_query_rows* q, const int32_t* q_lens, int32_t window) {
    return q->n == 1 && q_lens == nullptr && window == 0 && (q->num_heads == 1 || q->stride_h == c.head_dim) &&
           (c.batch == 1 || q->stride_b == static_cast<int64_t>(q->num_heads) * c.head_dim);
}

// ------------------------------------------------------------------- pages --
constexpr long long kMaxEntries = 1LL << 30;  // table entries, pages

struct PagesSpace {
    size_t page_a, page_b, seq_a, seq_b, old_table, moves, bytes;
};

PagesSpace pages_space(int32_t batch, int32_t num_pages, int32_t max_pages) {
    const size_t entries = static_cast<size_t>(batch) * max_pages, pages = static_cast<size_t>(num_pages);
    PagesSpace s{};
    size_t at = 256;
    auto take = [&at](size_t n) {
        const size_t here = at;
        at += align256(n);
        return here;
    };
    s.page_a = take(pages * 4);
    s.page_b = take(pages * 4);
    s.seq_a = take(static_cast<size_t>(batch) * 4);
    s.seq_b = take(static_cast<size_t>(batch) * 4);
    s.old_table = take(entries * 4);
    s.moves = take((entries > pages ? entries : pages) * sizeof(PageMove));
    s.bytes = at;
    return s;
}

bool pages_sizes(int32_t batch, int32_t num_pages, int32_t max_pages) {
    return batch >= 1 && num_pages >= 1 && num_pages <= kMaxEntries && max_pages >= 1 && static_cast<long long>(batch) * max_pages <= kMaxEntries;
}

tq_status pages_params(const Store& c, const int32_t* refs, const int32_t* held, void* workspace, size_t workspace_bytes, int32_t* status, PagesParams* p) {
    if (refs == nullptr || held == nullptr) return TQ_ERR_NULL;
    if (!pages_sizes(c.batch, c.map.num_pages, c.map.max_pages)) return TQ_ERR_SHAPE;
    if (static_cast<long long>(c.num_kv_heads) * c.map.page_tokens * c.head_dim * c.bits / 8 >= (1LL << 31)) return TQ_ERR_SHAPE;
    if (!aligned4(refs) || !aligned4(held) || !aligned4(c.map.block_table) || !aligned4(status)) return TQ_ERR_ALIGN;
    const PagesSpace sp = pages_space(c.batch, c.map.num_pages, c.map.max_pages);
    const tq_status s = check_workspace(workspace, workspace_bytes, sp.bytes);
    if (s != TQ_OK) return s;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    *p = PagesParams{};
    p->table = const_cast<int32_t*>(c.map.block_table);
    p->refs = const_cast<int32_t*>(refs);
    p->held = const_cast<int32_t*>(held);
    p->status = status;
    p->batch = c.batch;
    p->num_pages = c.map.num_pages;
    p->max_pages = c.map.max_pages;
    p->page_tokens = c.map.page_tokens;
    p->head = reinterpret_cast<int32_t*>(ws);
    p->page_a = reinterpret_cast<int32_t*>(ws + sp.page_a);
    p->page_b = reinterpret_cast<int32_t*>(ws + sp.page_b);
    p->seq_a = reinterpret_cast<int32_t*>(ws + sp.seq_a);
    p->seq_b = reinterpret_cast<int32_t*>(ws + sp.seq_b);
    p->old_table = reinterpret_cast<int32_t*>(ws + sp.old_table);
    p->moves = reinterpret_cast<PageMove*>(ws + sp.moves);
    p->codes[0] = c.k_codes;
    p->codes[1] = c.v_codes;
    p->sb[0] = c.k_scale;
    p->sb[1] = c.k_bias;
    p->sb[2] = c.v_scale;
    p->sb[3] = c.v_bias;
    p->num_kv_heads = c.num_kv_heads;
    p->head_dim = c.head_dim;
    p->bits = c.bits;
    return TQ_OK;
}

// The spans that every call has: refs, held, the workspace, the table, the status word, then the cache's arrays.
int common_spans(const Store& c, const PagesParams& p, size_t workspace_bytes, Span* s) {
    s[0] = {p.refs, 4ull * p.num_pages};
    s[1] = {p.held, 4ull * p.batch};
    s[2] = {p.head, workspace_bytes};
    s[3] = {p.table, 4ull * p.batch * p.max_pages};
    s[4] = {p.status, p.status != nullptr ? 4ull : 0ull};
    return 5 + arrays_of(c, s + 5);
}

}  // namespace

extern "C" {

size_t tq_chunk_workspace_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t n, int32_t max_seq_len) {
    return chunk_sizes(batch, hq, hkv, head_dim, n, max_seq_len) ? chunk_bytes(batch, hq, hkv, head_dim, n, max_seq_len) : 0;
}

tq_status tq_sdpa_chunk(const tq_kv_cache* cache, const tq_query_rows* q, const int32_t* q_lens, const int32_t* seq_lens, int32_t max_seq_len,
                        float attn_scale, int32_t window, uint32_t flags, void* workspace, size_t workspace_bytes, uint16_t* out,
                        int32_t* status, void* stream) {
    Store st;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK) s = check_chunk(st, q, q_lens, seq_lens, max_seq_len, window, flags, workspace, workspace_bytes, out, status);
    if (s != TQ_OK || q->n == 0) return s;
    if (is_decode(st, q, q_lens, window))
        return tq_sdpa_int4_decode_ex(cache, q->x, q->num_heads, seq_lens, max_seq_len, attn_scale, TQ_DEFAULT_CHUNK, flags & ~TQ_CHUNK_FULL, workspace, workspace_bytes,
                                      out, status, stream);
    return chunk(st, q, q_lens, seq_lens, max_seq_len, attn_scale, window, flags, workspace, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_paged_sdpa_chunk(const tq_paged_kv_cache* cache, const tq_query_rows* q, const int32_t* q_lens, const int32_t* seq_lens,
                              int32_t max_seq_len, float attn_scale, int32_t window, uint32_t flags, void* workspace,
                              size_t workspace_bytes, uint16_t* out, int32_t* status, void* stream) {
    Store st;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK) s = check_chunk(st, q, q_lens, seq_lens, max_seq_len, window, flags, workspace, workspace_bytes, out, status);
    if (s != TQ_OK || q->n == 0) return s;
    if (is_decode(st, q, q_lens, window))
        return tq_paged_sdpa_int4_decode(cache, q->x, q->num_heads, seq_lens, max_seq_len, attn_scale, TQ_DEFAULT_CHUNK, flags & ~TQ_CHUNK_FULL, workspace, workspace_bytes,
                                         out, status, stream);
    return chunk(st, q, q_lens, seq_lens, max_seq_len, attn_scale, window, flags, workspace, out, status, static_cast<cudaStream_t>(stream));
}

tq_status tq_chunk_timeout_selftest(const tq_kv_cache* cache, const tq_query_rows* q, const int32_t* seq_lens, int32_t max_seq_len, float attn_scale,
                                    uint32_t limit_us, int32_t copies, void* workspace, size_t workspace_bytes, uint16_t* out, int32_t* status,
                                    void* stream) {
    Store st;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK && status == nullptr) s = TQ_ERR_NULL;
    if (s == TQ_OK) s = check_chunk(st, q, nullptr, seq_lens, max_seq_len, 0, 0, workspace, workspace_bytes, out, status);
    if (s == TQ_OK && (limit_us < 1 || limit_us > 100000 || copies < 0)) s = TQ_ERR_SHAPE;
    if (s != TQ_OK || q->n == 0) return s;
    return chunk(st, q, nullptr, seq_lens, max_seq_len, attn_scale, 0, 0, workspace, out, status, static_cast<cudaStream_t>(stream), limit_us, copies);
}

size_t tq_pages_workspace_bytes(int32_t batch, int32_t num_pages, int32_t max_pages_per_seq) {
    return pages_sizes(batch, num_pages, max_pages_per_seq) ? pages_space(batch, num_pages, max_pages_per_seq).bytes : 0;
}

tq_status tq_pages_fork(const tq_paged_kv_cache* cache, int32_t* refs, int32_t* held, int32_t* lens, const int32_t* sources, void* workspace,
                        size_t workspace_bytes, int32_t* status, void* stream) {
    Store st;
    PagesParams p;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK && sources == nullptr) s = TQ_ERR_NULL;
    if (s == TQ_OK) s = pages_params(st, refs, held, workspace, workspace_bytes, status, &p);
    if (s != TQ_OK) return s;
    if (!aligned4(lens) || !aligned4(sources)) return TQ_ERR_ALIGN;
    Span sp[16];
    int n = common_spans(st, p, workspace_bytes, sp);
    // written: refs, held, workspace, table, status, lens
    sp[n++] = {sources, 4ull * p.batch};
    for (int i = n; i > 5; --i) sp[i] = sp[i - 1];
    sp[5] = {lens, lens != nullptr ? 4ull * p.batch : 0ull};
    ++n;
    if (clash(sp, n, 6)) return TQ_ERR_SHAPE;
    p.lens = lens;
    p.sources = sources;
    DeviceFacts* f = nullptr;
    s = device_facts(&f);
    return s != TQ_OK ? s : cuda_status(launch_pages_fork(p, f->sms, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_reserve(const tq_paged_kv_cache* cache, int32_t* refs, int32_t* held, const int32_t* start, int32_t n_rows, void* workspace,
                           size_t workspace_bytes, int32_t* status, void* stream) {
    Store st;
    PagesParams p;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK && start == nullptr) s = TQ_ERR_NULL;
    if (s == TQ_OK) s = pages_params(st, refs, held, workspace, workspace_bytes, status, &p);
    if (s != TQ_OK) return s;
    if (!aligned4(start)) return TQ_ERR_ALIGN;
    if (n_rows < 0) return TQ_ERR_SHAPE;
    if (n_rows > st.capacity) return TQ_ERR_CAPACITY;
    Span sp[16];
    int n = common_spans(st, p, workspace_bytes, sp);
    sp[n++] = {start, 4ull * p.batch};
    if (clash(sp, n, 11)) return TQ_ERR_SHAPE;
    if (n_rows == 0) return TQ_OK;
    p.start = start;
    p.n_rows = n_rows;
    DeviceFacts* f = nullptr;
    s = device_facts(&f);
    return s != TQ_OK ? s : cuda_status(launch_pages_reserve(p, f->sms, static_cast<cudaStream_t>(stream)));
}

tq_status tq_pages_compact(const tq_paged_kv_cache* cache, const int32_t* refs, const int32_t* held, int32_t* table_out, int32_t* refs_out,
                           int32_t* n_live, int32_t* moved, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    Store st;
    PagesParams p;
    tq_status s = store_of(cache, &st);
    if (s == TQ_OK && (table_out == nullptr || refs_out == nullptr || n_live == nullptr)) s = TQ_ERR_NULL;
    if (s == TQ_OK) s = pages_params(st, refs, held, workspace, workspace_bytes, status, &p);
    if (s != TQ_OK) return s;
    if (!aligned4(table_out) || !aligned4(refs_out) || !aligned4(n_live) || !aligned4(moved)) return TQ_ERR_ALIGN;
    // written: refs_out, table_out, n_live, moved, workspace, status, the cache's arrays
    Span sp[16] = {{refs_out, 4ull * p.num_pages}, {table_out, 4ull * p.batch * p.max_pages}, {n_live, 4ull},
                   {moved, moved != nullptr ? 4ull * p.num_pages : 0ull}, {p.head, workspace_bytes}, {status, status != nullptr ? 4ull : 0ull}};
    int n = 6 + arrays_of(st, sp + 6);
    const int refs_at = n, table_at = n + 1;
    sp[n++] = {refs, 4ull * p.num_pages};
    sp[n++] = {p.table, 4ull * p.batch * p.max_pages};
    sp[n++] = {held, 4ull * p.batch};
    if (clash(sp, n, 12, 0, refs_at, 1, table_at)) return TQ_ERR_SHAPE;
    p.table_out = table_out;
    p.refs_out = refs_out;
    p.n_live = n_live;
    p.moved = moved;
    DeviceFacts* f = nullptr;
    s = device_facts(&f);
    return s != TQ_OK ? s : cuda_status(launch_pages_compact(p, f->sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
