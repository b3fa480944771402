// pages.cu -- keeping account of the pages of a pool: forks of sequences (counted
// references to shared pages), pages for the next rows (the free ones of the
// lowest numbers, copies of shared pages that would be written) and compaction.
//
// The bookkeeping is integer work over tables of some thousand entries: bound by
// latency, so it is done by one CTA (its phases ordered by CTA barriers), and
// the copies of rows by a second launch over the whole device that reads the
// list of moves the first one left.  (32 beams forked and given room for a token: 12.2 us
// in three launches; half of 4,096 pages of 147 KB compacted: 55.0 us, 47 of them
// copies at 6.4 TB/s, 7 the list.)
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
// Largest table that a fork stages in one CTA's shared memory: one launch instead of two (32 x 65
// entries), but one CTA's reads and atomics (64 x 131 entries and the reservation behind
// them: 23.8 us in one CTA, 17.8 over the device when this was chosen).
constexpr int kForkEntries = 8192;
constexpr int kForkSeqs = kPlanThreads;

__device__ __forceinline__ void report(int32_t* status, int bit) {
    if (status != nullptr) atomicOr(status, bit);
}

__device__ __forceinline__ int clamp_held(const PagesParams& p, int held) {
    if (held >= 0 && held <= p.max_pages) return held;
    report(p.status, TQ_DEV_PAGE);
    return held < 0 ? 0 : p.max_pages;
}

// Whether a table entry names a page (else TQ_DEV_PAGE).
__device__ __forceinline__ bool is_page(const PagesParams& p, int page) {
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return true;
    report(p.status, TQ_DEV_PAGE);
    return false;
}

// Exclusive prefix sum over the CTA (kPlanThreads threads); total: the sum.
__device__ __forceinline__ int cta_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sums may still be read from the last call
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[kPlanThreads / 32 - 1];
    return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// ------------------------------------------------------------------- fork --
// One entry of the new table.
__device__ __forceinline__ int source_of(const PagesParams& p, int b) {
    const int s = p.sources[b];
    if (s >= -1 && s < p.batch) return s;
    report(p.status, TQ_DEV_SOURCE);
    return b;
}

__global__ void __launch_bounds__(kPlanThreads) fork_small_kernel(PagesParams p) {
    __shared__ int32_t old[kForkEntries];
    __shared__ int16_t from[kForkSeqs];
    __shared__ int32_t held[kForkSeqs];
    const int entries = p.batch * p.max_pages;
    // (up to kForkSeqs sequences: a thread each)
    int len = 0;
    if (static_cast<int>(threadIdx.x) < p.batch) {
        const int s = source_of(p, threadIdx.x);
        held[threadIdx.x] = clamp_held(p, p.held[threadIdx.x]);
        from[threadIdx.x] = static_cast<int16_t>(s);
        if (p.lens != nullptr && s >= 0) len = p.lens[s];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < entries; e += kPlanThreads) {
        const int b = e / p.max_pages, j = e - b * p.max_pages;
        const int page = p.table[e];
        old[e] = page;
        if (j < held[b] && is_page(p, page)) atomicSub(p.refs + page, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < entries; e += kPlanThreads) {
        const int b = e / p.max_pages, j = e - b * p.max_pages;
        const int s = from[b];
        int page = -1;
        if (s >= 0 && j < held[s]) {
            page = old[s * p.max_pages + j];
            if (is_page(p, page)) atomicAdd(p.refs + page, 1);
        }
        p.table[e] = page;
    }
    if (static_cast<int>(threadIdx.x) < p.batch) {
        const int s = from[threadIdx.x];
        p.held[threadIdx.x] = s < 0 ? 0 : held[s];
        if (p.lens != nullptr) p.lens[threadIdx.x] = len;
    }
}

// Tables past one CTA: the old state to the workspace, then the new one from it.
__global__ void __launch_bounds__(kCopyThreads) fork_release_kernel(PagesParams p) {
    const long long entries = static_cast<long long>(p.batch) * p.max_pages;
    for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
        const int b = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<long long>(b) * p.max_pages);
        const int page = p.table[e], held = clamp_held(p, p.held[b]);
        p.old_table[e] = page;
        if (j < held && is_page(p, page)) atomicSub(p.refs + page, 1);
        if (j == 0) {
            p.seq_a[b] = held;
            p.seq_b[b] = p.lens != nullptr ? p.lens[b] : 0;
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) fork_take_kernel(PagesParams p) {
    pdl_wait_primary();
    const long long entries = static_cast<long long>(p.batch) * p.max_pages;
    for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
        const int b = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<long long>(b) * p.max_pages);
        const int s = source_of(p, b), held = s < 0 ? 0 : p.seq_a[s];
        int page = -1;
        if (j < held) {
            page = p.old_table[static_cast<long long>(s) * p.max_pages + j];
            if (is_page(p, page)) atomicAdd(p.refs + page, 1);
        }
        p.table[e] = page;
        if (j == 0) {
            p.held[b] = held;
            if (p.lens != nullptr) p.lens[b] = s < 0 ? 0 : p.seq_b[s];
        }
    }
}

// ---------------------------------------------------------------- reserve --
// The entries [first, last] that sequence b's rows fall into, and how many it holds.
struct Range {
    int first, last, held;
};

__device__ __forceinline__ bool range_of(const PagesParams& p, int b, Range& r) {
    const int start = p.start[b];
    if (start < 0 || static_cast<long long>(start) + p.n_rows > static_cast<long long>(p.max_pages) * p.page_tokens) {
        report(p.status, TQ_DEV_WRITE_POS);
        return false;
    }
    r.first = start / p.page_tokens;
    r.last = static_cast<int>((static_cast<long long>(start) + p.n_rows - 1) / p.page_tokens);
    r.held = clamp_held(p, p.held[b]);
    return true;
}

// page_a counts the writers of each shared page, page_b holds the last of them.
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(PagesParams p) {
    __shared__ int warp_sums[32];
    __shared__ int n_moves;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kPlanThreads / 32;
    if (threadIdx.x == 0) n_moves = 0;
    // the shared pages that would be written (a warp per sequence, a lane per entry)
    for (int pass = 0; pass < 2; ++pass) {
        for (int b = warp; b < p.batch; b += kWarps) {
            Range r;
            if (!range_of(p, b, r)) continue;
            for (int j = r.first + lane; j <= r.last && j < r.held; j += 32) {
                const int page = p.table[static_cast<long long>(b) * p.max_pages + j];
                if (!is_page(p, page) || p.refs[page] <= 1) continue;
                if (pass == 0) {
                    p.page_a[page] = 0;
                    p.page_b[page] = -1;
                } else {
                    atomicAdd(p.page_a + page, 1);
                    atomicMax(p.page_b + page, b);
                }
            }
        }
        __syncthreads();
    }
    // a writer keeps the page when all that name it write and it is the last
    auto copies = [&](int b, const Range& r, int j, int& page) {
        if (j < r.first || j > r.last || j >= r.held) return false;
        page = p.table[static_cast<long long>(b) * p.max_pages + j];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) return false;
        const int refs = p.refs[page];
        return refs > 1 && !(__ldcg(p.page_a + page) == refs && __ldcg(p.page_b + page) == b);
    };
    for (int b = warp; b < p.batch; b += kWarps) {
        Range r;
        int wants = 0;
        if (range_of(p, b, r)) {
            for (int j0 = r.first; j0 <= r.last && j0 < r.held; j0 += 32) {
                int page;
                wants += __popc(__ballot_sync(0xffffffffu, copies(b, r, j0 + lane, page)));
            }
            if (r.last >= r.held) wants += r.last + 1 - r.held;
        }
        if (lane == 0) p.seq_a[b] = wants;
    }
    __syncthreads();
    // where each sequence's pages begin in the list of free ones
    long long carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int total;
        const int at = cta_scan(b < p.batch ? p.seq_a[b] : 0, warp_sums, total);
        // more than there are pages does not fit whatever the sum is
        if (b < p.batch) p.seq_a[b] = static_cast<int>(min(carry + at, 1LL << 30));
        carry += total;
    }
    const long long want = carry;
    if (want == 0) {
        if (threadIdx.x == 0) p.head[0] = 0;
        return;
    }
    // the lowest free pages, as many as wanted, into a list
    int found = 0;
    for (int q0 = 0; q0 < p.num_pages && found < want; q0 += kPlanThreads) {
        const int page = q0 + threadIdx.x;
        const bool free = page < p.num_pages && p.refs[page] == 0;
        int total;
        const int at = found + cta_scan(free ? 1 : 0, warp_sums, total);
        if (free && at < want) p.old_table[at] = page;
        found += total;
    }
    __syncthreads();
    if (found < want) {
        if (threadIdx.x == 0) {
            p.head[0] = 0;
            report(p.status, TQ_DEV_NO_PAGE);
        }
        return;
    }
    // hand them out: copies first, then the entries behind the held ones
    for (int b = warp; b < p.batch; b += kWarps) {
        Range r;
        if (!range_of(p, b, r)) continue;
        int at = p.seq_a[b];
        int32_t* row = p.table + static_cast<long long>(b) * p.max_pages;
        for (int j0 = r.first; j0 <= r.last && j0 < r.held; j0 += 32) {
            int page;
            const bool c = copies(b, r, j0 + lane, page);
            const unsigned mask = __ballot_sync(0xffffffffu, c);
            if (c) {
                const int fresh = p.old_table[at + __popc(mask & ((1u << lane) - 1))];
                const long long below = static_cast<long long>(p.start[b]) - static_cast<long long>(j0 + lane) * p.page_tokens;
                p.moves[atomicAdd(&n_moves, 1)] = {page, fresh, static_cast<int>(max(0LL, min(below, static_cast<long long>(p.page_tokens))))};
                row[j0 + lane] = fresh;
            }
            at += __popc(mask);
        }
        for (int j = r.held + lane; j <= r.last; j += 32) row[j] = p.old_table[at + j - r.held];
        __syncwarp();  // every lane has read the old count
        if (lane == 0 && r.last >= r.held) p.held[b] = r.last + 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < want; i += kPlanThreads) p.refs[p.old_table[i]] = 1;
    for (int i = threadIdx.x; i < n_moves; i += kPlanThreads) atomicSub(p.refs + p.moves[i].src, 1);
    if (threadIdx.x == 0) p.head[0] = n_moves;
}

// The same for up to 128 sequences whose rows fall into at most 32 entries each (a
// step's): what each warp reads of its sequences stays in registers, wants and free
// pages in shared memory.  (32 beams, caches cold: 6 us instead of 11.)
constexpr int kSmallSeqs = 128;

__global__ void __launch_bounds__(kPlanThreads) reserve_small_kernel(PagesParams p) {
    constexpr int kWarps = kPlanThreads / 32, kEach = kSmallSeqs / kWarps;
    __shared__ int warp_sums[32], offset[kSmallSeqs], list[kPlanThreads], n_moves, total;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first_refs = static_cast<int>(threadIdx.x) < p.num_pages ? p.refs[threadIdx.x] : 1;
    if (threadIdx.x == 0) n_moves = 0;
    Range r[kEach];
    bool in[kEach], copied[kEach];
    int page[kEach], refs[kEach], start[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int b = warp + k * kWarps;
        in[k] = b < p.batch && range_of(p, b, r[k]);
        start[k] = in[k] ? p.start[b] : 0;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int j = in[k] ? r[k].first + lane : 0;
        page[k] = in[k] && j <= r[k].last && j < r[k].held ? p.table[static_cast<long long>(warp + k * kWarps) * p.max_pages + j] : -1;
        // (no entry at all is not an entry outside the pool)
        if (in[k] && j <= r[k].last && j < r[k].held && !is_page(p, page[k])) page[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        refs[k] = page[k] >= 0 ? p.refs[page[k]] : 0;
        if (refs[k] > 1) {
            p.page_a[page[k]] = 0;
            p.page_b[page[k]] = -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (refs[k] > 1) {
            atomicAdd(p.page_a + page[k], 1);
            atomicMax(p.page_b + page[k], warp + k * kWarps);
        }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int b = warp + k * kWarps;
        copied[k] = refs[k] > 1 && !(__ldcg(p.page_a + page[k]) == refs[k] && __ldcg(p.page_b + page[k]) == b);
        const int copies = __popc(__ballot_sync(0xffffffffu, copied[k]));
        if (lane == 0) offset[b] = in[k] ? copies + (r[k].last >= r[k].held ? r[k].last + 1 - r[k].held : 0) : 0;
    }
    __syncthreads();
    if (warp == 0) {
        // (sums: at most 128 sequences of 2^30 entries in all)
        int v[kEach], sum = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            v[k] = offset[lane * kEach + k];
            sum += v[k];
        }
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) total = x;
        x -= sum;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            offset[lane * kEach + k] = x;
            x += v[k];
        }
    }
    __syncthreads();
    const int want = total;
    if (want == 0) {
        if (threadIdx.x == 0) p.head[0] = 0;
        return;
    }
    int32_t* fresh = want <= kPlanThreads ? list : p.old_table;
    int found = 0;
    for (int q0 = 0; q0 < p.num_pages && found < want; q0 += kPlanThreads) {
        const int q = q0 + threadIdx.x;
        const bool free = q < p.num_pages && (q0 == 0 ? first_refs : p.refs[q]) == 0;
        int sum;
        const int at = found + cta_scan(free ? 1 : 0, warp_sums, sum);
        if (free && at < want) fresh[at] = q;
        found += sum;
    }
    __syncthreads();
    if (found < want) {
        if (threadIdx.x == 0) {
            p.head[0] = 0;
            report(p.status, TQ_DEV_NO_PAGE);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (!in[k]) continue;
        const int b = warp + k * kWarps;
        int at = offset[b];
        int32_t* row = p.table + static_cast<long long>(b) * p.max_pages;
        const unsigned mask = __ballot_sync(0xffffffffu, copied[k]);
        if (copied[k]) {
            const int to = fresh[at + __popc(mask & ((1u << lane) - 1))], j = r[k].first + lane;
            const long long below = static_cast<long long>(start[k]) - static_cast<long long>(j) * p.page_tokens;
            p.moves[atomicAdd(&n_moves, 1)] = {page[k], to, static_cast<int>(max(0LL, min(below, static_cast<long long>(p.page_tokens))))};
            row[j] = to;
            atomicSub(p.refs + page[k], 1);
        }
        at += __popc(mask);
        for (int j = r[k].held + lane; j <= r[k].last; j += 32) row[j] = fresh[at + j - r[k].held];
        if (lane == 0 && r[k].last >= r[k].held) p.held[b] = r[k].last + 1;
    }
    for (int i = threadIdx.x; i < want; i += kPlanThreads) p.refs[fresh[i]] = 1;
    __syncthreads();
    if (threadIdx.x == 0) p.head[0] = n_moves;
}

// ---------------------------------------------------------------- compact --
// page_a: for a moved page its place in the list of moves, for the others not set.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesParams p) {
    __shared__ int warp_sums[32];
    int live = 0;
    for (int q = threadIdx.x; q < p.num_pages; q += kPlanThreads) live += p.refs[q] > 0 ? 1 : 0;
    int n;
    cta_scan(live, warp_sums, n);
    int holes = 0, late = 0;
    for (int q0 = 0; q0 < p.num_pages; q0 += kPlanThreads) {
        const int page = q0 + threadIdx.x;
        const bool used = page < p.num_pages && p.refs[page] > 0;
        const bool hole = page < n && !used, moves = page >= n && used;
        int total;
        // both in one scan: no more than 2^15 of either in a step
        const int at = cta_scan((hole ? 1 : 0) | (moves ? 1 << 16 : 0), warp_sums, total);
        if (hole) p.moves[holes + (at & 0xffff)].dst = page;
        if (moves) {
            p.moves[late + (at >> 16)].src = page;
            p.page_a[page] = late + (at >> 16);
        }
        holes += total & 0xffff;
        late += total >> 16;
        if (page < p.num_pages && p.moved != nullptr) p.moved[page] = used ? page : -1;
    }
    __syncthreads();
    // refs_out may be refs: first what stays and what moves to a hole, then the zeros
    for (int i = threadIdx.x; i < late; i += kPlanThreads) {
        p.moves[i].rows = p.page_tokens;
        p.refs_out[p.moves[i].dst] = p.refs[p.moves[i].src];
        if (p.moved != nullptr) p.moved[p.moves[i].src] = p.moves[i].dst;
    }
    if (p.refs_out != p.refs)
        for (int q = threadIdx.x; q < n; q += kPlanThreads)
            if (p.refs[q] > 0) p.refs_out[q] = p.refs[q];
    __syncthreads();
    for (int q = n + threadIdx.x; q < p.num_pages; q += kPlanThreads) p.refs_out[q] = 0;
    if (threadIdx.x == 0) {
        p.head[0] = late;
        p.head[1] = n;
        *p.n_live = n;
    }
}

// ------------------------------------------------------------------- rows --
// `bytes` bytes by the CTA's threads: 16 at a time, four of a thread's in flight, the
// last ones two at a time.
__device__ __forceinline__ void copy_span(uint8_t* dst, const uint8_t* src, int bytes) {
    const int vecs = bytes >> 4;
    uint4* d = reinterpret_cast<uint4*>(dst);
    const uint4* s = reinterpret_cast<const uint4*>(src);
    int i = threadIdx.x;
    for (; i + 3 * kCopyThreads < vecs; i += 4 * kCopyThreads) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __ldcs(s + i + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k) __stcs(d + i + k * kCopyThreads, v[k]);
    }
    for (; i < vecs; i += kCopyThreads) __stcs(d + i, __ldcs(s + i));
    for (i = vecs * 8 + threadIdx.x; i < bytes >> 1; i += kCopyThreads)
        reinterpret_cast<uint16_t*>(dst)[i] = reinterpret_cast<const uint16_t*>(src)[i];
}

// The listed moves.  A unit is one of the six arrays of a page, or (heads: first rows
// of a page, few moves) of one head of it.
template <bool HEADS>
__device__ __forceinline__ void copy_moves(const PagesParams& p) {
    const int n = p.head[0], each = HEADS ? p.num_kv_heads : 1;
    const int cw = p.head_dim * p.bits / 8, sw = p.head_dim / kGroup * 2;
    const long long codes = 2LL * n * each;  // codes first: most of the bytes are theirs
    for (long long u = blockIdx.x; u < 3 * codes; u += gridDim.x) {
        const bool scale = u >= codes;
        const long long v = (scale ? u - codes : u) / each;
        const int h = HEADS ? static_cast<int>(u % each) : 0;
        const int a = scale ? static_cast<int>(v % 4) : static_cast<int>(v % 2), width = scale ? sw : cw;
        const PageMove m = p.moves[scale ? v / 4 : v / 2];
        uint8_t* at = scale ? reinterpret_cast<uint8_t*>(p.sb[a]) : p.codes[a];
        const long long head = static_cast<long long>(p.page_tokens) * width, page = head * p.num_kv_heads;
        // (a page's codes are at most 2^31 bytes: its host check)
        copy_span(at + m.dst * page + h * head, at + m.src * page + h * head, HEADS ? m.rows * width : static_cast<int>(page));
    }
}

__global__ void __launch_bounds__(kCopyThreads) move_rows_kernel(PagesParams p) {
    pdl_wait_primary();
    copy_moves<true>(p);
}

__global__ void __launch_bounds__(kCopyThreads) compact_rows_kernel(PagesParams p) {
    pdl_wait_primary();
    const int n = p.head[1];
    const long long step = static_cast<long long>(gridDim.x) * kCopyThreads, first = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x;
    const long long entries = static_cast<long long>(p.batch) * p.max_pages;
    for (long long e = first; e < entries; e += step) {
        const int b = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<long long>(b) * p.max_pages);
        int page = p.table[e];
        // (an entry whose page is counted free keeps its number: page_a holds nothing for it)
        if (j < clamp_held(p, p.held[b]) && is_page(p, page) && page >= n) {
            const int k = p.page_a[page];
            if (static_cast<unsigned>(k) < static_cast<unsigned>(p.head[0]) && p.moves[k].src == page) page = p.moves[k].dst;
        }
        p.table_out[e] = page;
    }
    copy_moves<false>(p);
}

}  // namespace

cudaError_t launch_pages_fork(const PagesParams& p, int sms, cudaStream_t stream) {
    const long long entries = static_cast<long long>(p.batch) * p.max_pages;
    if (entries <= kForkEntries && p.batch <= kForkSeqs) {
        fork_small_kernel<<<1, kPlanThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const long long ctas = (entries + kCopyThreads - 1) / kCopyThreads;
    const unsigned grid = static_cast<unsigned>(ctas < 8LL * sms ? ctas : 8LL * sms);
    fork_release_kernel<<<grid, kCopyThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(fork_take_kernel, grid, kCopyThreads, stream, p);
}

cudaError_t launch_pages_reserve(const PagesParams& p, int sms, cudaStream_t stream) {
    // the most entries that a sequence's rows fall into (rows and a page may pass 2^31 together)
    const long long entries = (static_cast<long long>(p.n_rows) + p.page_tokens - 2) / p.page_tokens + 1;
    if (p.batch <= kSmallSeqs && entries <= 32)
        reserve_small_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    else
        reserve_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // no more units of work than heads of the arrays of the pages that the rows touch
    const long long units = 6LL * p.num_kv_heads * p.batch * entries;
    return launch_after(move_rows_kernel, static_cast<unsigned>(units < 4LL * sms ? units : 4LL * sms), kCopyThreads, stream, p);
}

cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream) {
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(compact_rows_kernel, static_cast<unsigned>(8 * sms), kCopyThreads, stream, p);
}

}  // namespace tq
