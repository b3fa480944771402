// chunk.cu -- attention of several query rows per sequence over the cache: a
// chunk of new tokens in causal order (optionally the last `window` tokens
// only), or every row over the whole sequence.  For row r = (token i, head g) of
// (sequence b, kv head h), r = i * G + g:
//   out_r = sum_t p_t V_t / sum_t p_t,  p_t = 2^(c q_r.K_t - m_r),  lo_i <= t < hi_i,
// with c = attn_scale log2(e) and m_r a running maximum less seven.  Rows of all the heads
// that share a kv head are rows of one matrix, so every cached key and value is
// unpacked once for 256 of them.
//
// A CTA takes 256 rows (two tiles of 128, the M of a tcgen05.mma; one tile at
// head_dim 256, whose output fills half of TMEM) and a run of the keys they see, in
// tiles of 128 (64 at head_dim 256):
//   a copying warp    brings codes, scales and biases into a ring (bulk copies)
//   unpacking warps   turn them into fp16 operands in shared memory, laid out as
//                     128-byte rows with the 128-byte swizzle: keys are then a
//                     K-major operand and values an N-major one, in the same layout
//   two MMA warps     S = Q K^T and O += P V, S, P and O in TMEM
//   softmax warps     a thread a row: maximum, 2^x, P as fp16, sum; no shuffles
// S is read into registers as soon as it is there, so that one place for it serves both
// row tiles in turn and their scores run ahead of the softmax.  Up to 128 rows (a few
// tokens) make one tile; the two accumulators then take every other tile of keys and are
// merged in the end.  P starts at 2^7, and O is rescaled only when a row's maximum grows by
// more than 2^8 (the published conditional rescaling of online softmax), which is rare
// after the first tiles: P uses fp16's range up to 2^15, so that weights down to 2^-21 of a
// row's largest keep all their bits and those above 2^-32 of it are more than zero.  (With P
// from 1 up, a key that took most of a row's weight left nothing of the others 25
// powers of two below it, however many.)  Where there are few items
// for the SMs their keys are cut into runs, whose states a second kernel merges.
//
// An accumulator takes 8,192 keys at most before it is emptied into sums in memory: the
// tensor cores' sums are not rounded to nearest, and what they lose grows with the length.
//
// Rounding: cached values enter the products as fp16 (half a step of 2^-11, what
// the tensor core takes), P as fp16 (the sums take it unrounded); S, O, maxima and sums
// are fp32.
//
// What bounds it (GB300, 64 query and 8 kv heads of 128, int4): for long chunks the
// turn of the one place for S (a product of 512 cycles, then some 800 of commits, waits
// and reads until it is free again) and the instructions of softmax and unpacking (65 %
// of the issue slots): 2,048 tokens over 65,536 in 2.73 ms, 1.59 PFLOP/s (3.11 ms and 1.39
// where many such calls bring the clocks down by power); a prompt of 8,192
// in 0.84 ms, 1.32 PFLOP/s with 16,000 cycles of start and end in each CTA.  For eight
// tokens over 131,072 it is the unpacking (2,100 cycles a tile of 128 keys, 800 of HBM
// time): 73.1 us, of which 23 are what the cache's bytes take.
#include <stddef.h>

#include "tq_device.cuh"
#include "tq_hadamard.cuh"
#include "tq_internal.h"
#include "tq_tcgen05.cuh"

namespace tq {

namespace {

constexpr int kThreads = 640;       // 8 softmax warps, 8 that unpack, 2 that issue products, one that copies
constexpr int kRowTile = 128;
constexpr float kHead = 7.f;  // log2 of a row's largest P when its maximum is new
constexpr float kLazy = 8.f;  // log2 of how far P may grow from there before O is rescaled
static_assert(kHead + kLazy <= 15.f, "P in fp16");

template <int D, int BITS>
struct Cfg {
    static constexpr int kStreams = D == 256 ? 1 : 2;         // softmax warpgroups, output accumulators
    static constexpr int kTile = D == 256 ? 64 : 128;         // keys
    static constexpr int kSoftmax = kStreams * 128;           // softmax threads: one for each row
    static constexpr int kUnpackWarp = 8;                     // first unpacking warp
    static constexpr int kUnpackWarps = 8;
    static constexpr int kBlocks = D / 64;                    // blocks of 64 channels: 128-byte rows
    static constexpr int kSlot = kTile * D * 2;               // one unpacked tile of keys or values
    static constexpr int kSlots = D == 64 ? 6 : 3;
    static constexpr int kCodes = kTile * D * BITS / 8;
    static constexpr int kScales = kTile * kBlocks * 2;       // scales (and as many biases) of a tile
    static constexpr int kEntry = kCodes + 2 * kScales;
    static constexpr int kChain = kChunkChainKeys / kTile;    // turns of an accumulator between its emptyings
    static_assert((kChain & (kChain - 1)) == 0, "a mask tells where a chain begins");
    static constexpr int kRing = D == 64 ? 6 : (BITS == 8 ? 3 : 6);
    static constexpr int kQ = kStreams * kRowTile * D * 2;
    // one row tile: the other's place holds more of the ring (few rows: what bounds is how
    // many bytes are on their way)
    static constexpr int kMoreRing = kStreams == 2 ? kRowTile * D * 2 / kEntry : 0;
    static_assert(kRing + kMoreRing <= 10, "barriers");
    static constexpr int kSmem = 1024 + kQ + kSlots * kSlot + kRing * kEntry;
    static_assert(kQ + kSlots * kSlot >= kStreams * D * (kRowTile + 1) * 4, "rows on their way out");
    // TMEM columns: scores (one place for both accumulators at head_dim 128, else two),
    // weights P of either parity as fp16, outputs
    static constexpr int kPlaces = D == 128 ? 1 : 2;
    static constexpr uint32_t kS1 = D == 64 ? 384 : 64;       // the second place for scores
    static constexpr uint32_t kP = 128, kPStep = kTile / 2;
    static constexpr uint32_t kO = 256;
    static_assert(kSmem + 6144 <= 232448, "shared memory of a CTA");
    static_assert(kO + kStreams * D <= (D == 64 ? kS1 : 512u) && kP + 2 * kPStep <= kO && kTile <= 128, "TMEM");
};

struct Bars {
    uint64_t ring_full[10], ring_empty[10], slot_full[6], slot_empty[6];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_full, drain[2];
    uint32_t tmem;
    int32_t abort;
    float max[kRowTile], sum[kRowTile];  // the second accumulator's, where both are of one row tile
};

// Addresses of the barriers from that of the first.  (Each role takes the first one's
// once, in a way that the compiler cannot repeat: left to it, it forms a shared
// variable's address anew wherever it is used, from a special register that takes
// tens of cycles to read, which between two products is time lost.)
enum : uint32_t {
    kRingFull = 0,
    kRingEmpty = 10 * 8,
    kSlotFull = 20 * 8,
    kSlotEmpty = 26 * 8,
    kSFull = 32 * 8,
    kSFree = 34 * 8,
    kPFull = 36 * 8,
    kPvDone = 38 * 8,
    kQFull = 40 * 8,
    kDrain = 41 * 8,
    kTmemAt = 43 * 8,
    kAbort = 43 * 8 + 4,
};
__device__ __forceinline__ uint32_t fixed(uint32_t x) {
    asm volatile("" : "+r"(x));
    return x;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Token and head of row `flat` of a (sequence, kv head): flat / group_q (rows fewer than 2^28 * 8).
__device__ __forceinline__ void row_of(const ChunkParams& p, int flat, int& i, int& g) {
    i = p.group_magic == 0 ? flat : static_cast<int>(__umulhi(static_cast<unsigned>(flat), p.group_magic) >> p.group_shift);
    g = flat - i * p.group_q;
}

// What a CTA works on.
struct Work {
    int b, h;
    int part;               // where partial states go (-1: the output is written)
    int row0, rows;         // first row, valid rows from it on (up to kStreams * 128)
    int ql, len;
    int klo, khi;           // the keys that any of the rows sees
    int tile0, tiles;       // this CTA's tiles of keys
};

__device__ __forceinline__ int first_key(const ChunkParams& p, int i, int ql, int len) {
    const int pos = len - ql + i;
    return !p.full && p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
}
__device__ __forceinline__ int end_key(const ChunkParams& p, int i, int ql, int len) {
    if (p.full) return len;
    const int pos = len - ql + i;
    return pos + 1 > 0 ? pos + 1 : 0;
}

template <int TILE>
__device__ __forceinline__ bool find_work(const ChunkParams& p, int rows_per_item, Work& w) {
    // The last rows' items first (in causal order they see the most keys), the first
    // p.whole of them whole, the others in n_splits runs.
    int id = blockIdx.x, split = 0, splits = 1;
    w.part = -1;
    if (id >= p.whole) {
        w.part = id - p.whole;
        id = p.whole + w.part / p.n_splits;
        split = w.part - (id - p.whole) * p.n_splits;
        splits = p.n_splits;
        if (splits == 1) w.part = -1;
    }
    const int per = p.batch * p.num_kv_heads, above = id / per, bh = id - above * per, m = p.m_items - 1 - above;
    w.b = bh / p.num_kv_heads;
    w.h = bh - w.b * p.num_kv_heads;
    int len = p.seq_lens[w.b], ql = p.q_lens != nullptr ? p.q_lens[w.b] : p.n;
    if (len < 0 || len > p.max_seq_len || ql < 0 || ql > p.n) {
        if (p.status != nullptr && threadIdx.x == 0) atomicOr(p.status, TQ_DEV_SEQ_LEN);
        len = min(max(len, 0), p.max_seq_len);
        ql = min(max(ql, 0), p.n);
    }
    w.len = len;
    w.ql = ql;
    w.row0 = m * rows_per_item;
    w.rows = min(rows_per_item, ql * p.group_q - w.row0);
    if (w.rows <= 0) return false;
    int i0, i1, g;
    row_of(p, w.row0, i0, g);
    row_of(p, w.row0 + w.rows - 1, i1, g);
    w.klo = first_key(p, i0, ql, len);
    w.khi = end_key(p, i1, ql, len);
    w.tile0 = w.klo / TILE;
    const int all = w.khi > w.klo ? (w.khi + TILE - 1) / TILE - w.tile0 : 0;
    const int t0 = static_cast<int>(static_cast<long long>(all) * split / splits);
    w.tiles = static_cast<int>(static_cast<long long>(all) * (split + 1) / splits) - t0;
    w.tile0 += t0;
    return true;
}

// Entry e of the ring and of the slots: the keys or the values of tile `tile`.  The
// next keys come ahead of the values (K0 K1 V0 K2 V1 ... V_last).
__device__ __forceinline__ bool entry_of(int e, int tiles, int& tile) {
    if (e == 0) {
        tile = 0;
        return false;
    }
    if (e & 1) {
        tile = (e + 1) >> 1;
        if (tile < tiles) return false;
        tile = tiles - 1;
        return true;
    }
    tile = (e >> 1) - 1;
    return true;
}
__device__ __forceinline__ int key_entry(int tile) { return tile == 0 ? 0 : 2 * tile - 1; }
__device__ __forceinline__ int value_entry(int tile, int tiles) { return tile == tiles - 1 ? 2 * tiles - 1 : 2 * tile + 2; }

// Whether a phase is over; the hardware holds the warp for a while if it is not.
// (With a time limit of its own, as mbar_try_wait asks for, the wait becomes a loop that
// polls and sleeps: 350 sleeps and 700 polls a tile of keys, in the way of the warps that work.)
__device__ __forceinline__ bool over(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Microseconds of a sort (1,024 ns each), never 0.
__device__ __forceinline__ uint32_t globaltimer_us() { return static_cast<uint32_t>(globaltimer_ns() >> 10) | 1u; }

// Waits for a phase of the barrier at `bar`; false when it took too long or another warp
// has given up.  All lanes of a warp are here together, and get one answer: where a lane
// gave up as its neighbours went on, these would wait for it at their next warp-wide
// instruction.  (The timer is read rarely: that takes longer than most waits.)
__device__ __forceinline__ bool wait(const ChunkParams& p, uint32_t bars, uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, over(bars + bar, parity))) return true;
    uint32_t since = 0;
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, over(bars + bar, parity))) return true;
        if ((it & 63u) == 0) {
            bool stop = lds32(bars + kAbort) != 0;
            if ((it & 1023u) == 0) {
                const uint32_t now = globaltimer_us();
                if (since == 0) since = now;
                if (now - since > p.limit_us) {
                    stop = true;
                    asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(bars + kAbort) : "memory");
                    if (p.status != nullptr) atomicOr(p.status, TQ_DEV_TIMEOUT);
                }
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}

// ------------------------------------------------------------------ loader --
// Where entry r of the ring lies.
template <int D, int BITS>
__device__ __forceinline__ uint32_t ring_at(uint32_t ring, uint32_t more, int r) {
    using C = Cfg<D, BITS>;
    return r < C::kRing ? ring + r * C::kEntry : more + (r - C::kRing) * C::kEntry;
}

// One warp: its first three lanes copy an entry's codes, scales and biases.
template <int D, int BITS>
__device__ __forceinline__ void load_role(const ChunkParams& p, const Work& w, uint32_t ring, uint32_t more, int ring_entries, uint32_t bars) {
    using C = Cfg<D, BITS>;
    const uint64_t policy = policy_evict_first();
    const int lane = threadIdx.x & 31;
    const uint32_t width = lane == 0 ? D * BITS / 8 : C::kBlocks * 2, offset = lane == 0 ? 0 : (lane == 1 ? C::kCodes : C::kCodes + C::kScales);
    const uint8_t* keys = lane == 0 ? p.k_codes : reinterpret_cast<const uint8_t*>(lane == 1 ? p.k_scale : p.k_bias);
    const uint8_t* values = lane == 0 ? p.v_codes : reinterpret_cast<const uint8_t*>(lane == 1 ? p.v_scale : p.v_bias);
    int r = 0, issued = 0;
    uint32_t parity = 1;
    bool ok = true;
    auto issue = [&](const uint8_t* from, int tile, long long row) {
        if (issued == p.copies || !wait(p, bars, kRingEmpty + r * 8, parity)) return false;
        const int rows = min(C::kTile, (w.khi - (w.tile0 + tile) * C::kTile + 15) & ~15);  // capacities are whole 16s
        const uint32_t bar = bars + kRingFull + r * 8;
        if (lane == 0) asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(rows * (D * BITS / 8 + C::kBlocks * 4)) : "memory");
        __syncwarp();
        if (lane < 3)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                             ring_at<D, BITS>(ring, more, r) + offset),
                         "l"(from + row * width), "r"(rows * width), "r"(bar), "l"(policy)
                         : "memory");
        ++issued;
        if (++r == ring_entries) {
            r = 0;
            parity ^= 1;
        }
        return true;
    };
    // rows of the next tile are looked up (a table entry's latency) ahead of its copies
    long long row = 0, next = w.tiles > 0 ? kv_row(p.map, p.num_kv_heads, w.b, w.h, w.tile0 * C::kTile, p.status) : 0;
#pragma unroll 1
    for (int j = -1; j < w.tiles && ok; ++j) {
        long long after = 0;
        if (j + 2 < w.tiles) after = kv_row(p.map, p.num_kv_heads, w.b, w.h, (w.tile0 + j + 2) * C::kTile, p.status);
        if (j + 1 < w.tiles) ok = issue(keys, j + 1, next);
        if (j >= 0 && ok) ok = issue(values, j, row);
        row = next;
        next = after;
    }
    // the copies in flight land before the CTA leaves (also where other warps have given up)
    for (int k = max(0, issued - ring_entries); k < issued; ++k)
        for (int it = 0; it < 1 << 20 && !over(bars + kRingFull + k % ring_entries * 8, (k / ring_entries) & 1); ++it) {
        }
}

// ---------------------------------------------------------------- unpacking --
// Eight codes as four pairs of fp16.  int4: pairs (0,4), (1,5), (2,6), (3,7) of a
// word, the order that shifts and masks give; queries and outputs follow it.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

template <int BITS>
__device__ __forceinline__ void unpack8(uint32_t w0, uint32_t w1, __half2 (&c)[4]) {
    auto h2 = [](uint32_t x) { return *reinterpret_cast<__half2*>(&x); };
    const __half2 k1024 = __floats2half2_rn(1024.f, 1024.f), k64 = __floats2half2_rn(64.f, 64.f);
    if (BITS == 4) {
        // a nibble in the low bits of 0x6400 counts from 1,024 on, four bits up in 0x5400 from 64 on
        const uint32_t hi = w0 >> 8;
        c[0] = __hsub2(h2(and_or(w0, 0x000f000fu, 0x64006400u)), k1024);
        c[1] = __hsub2(h2(and_or(w0, 0x00f000f0u, 0x54005400u)), k64);
        c[2] = __hsub2(h2(and_or(hi, 0x000f000fu, 0x64006400u)), k1024);
        c[3] = __hsub2(h2(and_or(hi, 0x00f000f0u, 0x54005400u)), k64);
    } else {
        c[0] = __hsub2(h2(__byte_perm(w0, 0x64646464u, 0x4140)), k1024);
        c[1] = __hsub2(h2(__byte_perm(w0, 0x64646464u, 0x4342)), k1024);
        c[2] = __hsub2(h2(__byte_perm(w1, 0x64646464u, 0x4140)), k1024);
        c[3] = __hsub2(h2(__byte_perm(w1, 0x64646464u, 0x4342)), k1024);
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ __half lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return __ushort_as_half(v);
}
__device__ __forceinline__ void sts128(uint32_t at, const __half2 (&h)[4]) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(h);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// A thread takes the same 16-byte piece of every 2^n-th key's codes: where its
// outputs go, and in which order, is the same for all of them.
template <int D, int BITS>
__device__ __forceinline__ void unpack_role(const ChunkParams& p, const Work& w, uint32_t ring, uint32_t more, int ring_entries, uint32_t slots, uint32_t bars) {
    using C = Cfg<D, BITS>;
    constexpr int kUnits = BITS == 4 ? 4 : 2;             // 16-byte pieces of fp16 that 16 bytes of codes give
    constexpr int kChunks = D * BITS / 8 / 16;            // 16-byte pieces of codes per key
    constexpr int kT = C::kUnpackWarps * 32;
    constexpr int kKeys = kT / kChunks;                   // keys from one piece of a thread to its next
    constexpr int kIts = C::kTile / kKeys;
    static_assert(kKeys % 8 == 0 && kIts * kKeys == C::kTile, "pieces of a thread");
    const int tid = threadIdx.x - C::kUnpackWarp * 32, lane = threadIdx.x & 31;
    const int t = tid / kChunks, ck = tid % kChunks, g = ck * kUnits / 8, u0 = ck * kUnits % 8;
    // eight lanes write eight different 16-byte columns: pieces of other blocks are
    // taken in another order
    const int x = BITS == 4 ? (D == 128 ? g * 2 : (D == 256 ? g : 0)) : g & 1;
    uint32_t to[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) to[j] = slots + g * (C::kTile * 128) + t * 128 + (((u0 + (j ^ x)) ^ (t & 7)) << 4);
    auto in_order = [x](const uint4& word, uint32_t (&v)[4]) {
        v[0] = word.x, v[1] = word.y, v[2] = word.z, v[3] = word.w;
        auto swap = [&v](int a, int b) {
            const uint32_t y = v[a];
            v[a] = v[b];
            v[b] = y;
        };
        if (BITS == 4 && D == 256 && (x & 1)) swap(0, 1), swap(2, 3);
        if (D >= 128 && (BITS == 4 ? (x & 2) != 0 : x != 0)) swap(0, 2), swap(1, 3);
    };
    const uint32_t from = tid * 16, from_scale = C::kCodes + (t * C::kBlocks + g) * 2;
    int r = 0, s = 0;
    uint32_t r_parity = 0, s_parity = 1;
#pragma unroll 1
    for (int e = 0; e < 2 * w.tiles; ++e) {
        if (!wait(p, bars, kRingFull + r * 8, r_parity)) return;
        if (!wait(p, bars, kSlotEmpty + s * 8, s_parity)) return;  // (a fresh barrier's phase before the first is over)
        int tile;
        const bool value = entry_of(e, w.tiles, tile);
        const int t0 = (w.tile0 + tile) * C::kTile;
        const uint32_t at = ring_at<D, BITS>(ring, more, r), src = at + from, src_scale = at + from_scale, dst = s * C::kSlot;
        uint4 word[kIts];
        __half sc[kIts], bi[kIts];
        // values past fp16's range, scales or biases that are no numbers, keys that no row sees: apart
        bool odd = t0 < w.klo || t0 + C::kTile > w.khi;
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
            word[it] = lds128(src + it * kT * 16);
            sc[it] = lds16(src_scale + it * kKeys * C::kBlocks * 2);
            bi[it] = lds16(src_scale + C::kScales + it * kKeys * C::kBlocks * 2);
            odd = odd || !(__hfma(__habs(sc[it]), __float2half_rn(BITS == 4 ? 15.f : 255.f), __habs(bi[it])) <= __float2half_rn(65504.f));
        }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int it = 0; it < kIts; ++it) {
                const uint4 again = lds128(src + it * kT * 16);
                const float fs = __half2float(lds16(src_scale + it * kKeys * C::kBlocks * 2)),
                            fb = __half2float(lds16(src_scale + C::kScales + it * kKeys * C::kBlocks * 2));
                const int key = t0 + t + it * kKeys;
                const bool none = key < w.klo || key >= w.khi || (value && !(fabsf(fs) <= 65504.f && fabsf(fb) <= 65504.f));
                uint32_t v[4];
                in_order(again, v);
#pragma unroll
                for (int j = 0; j < kUnits; ++j) {
                    __half2 h[4];
                    unpack8<BITS>(v[BITS == 4 ? j : 2 * j], v[BITS == 4 ? j : 2 * j + 1], h);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = __half22float2(h[k]);
                        h[k] = none ? __floats2half2_rn(0.f, 0.f)
                                    : __floats2half2_rn(fminf(fmaxf(fmaf(f.x, fs, fb), -65504.f), 65504.f), fminf(fmaxf(fmaf(f.y, fs, fb), -65504.f), 65504.f));
                    }
                    sts128(dst + to[j] + it * kKeys * 128, h);
                }
            }
        } else {
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                uint32_t v[4];
                in_order(word[it], v);
                const __half2 s2 = __half2half2(sc[it]), b2 = __half2half2(bi[it]);
#pragma unroll
                for (int j = 0; j < kUnits; ++j) {
                    __half2 h[4];
                    unpack8<BITS>(v[BITS == 4 ? j : 2 * j], v[BITS == 4 ? j : 2 * j + 1], h);
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = __hfma2(h[k], s2, b2);
                    sts128(dst + to[j] + it * kKeys * 128, h);
                }
            }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            arrive(bars + kRingEmpty + r * 8);
            arrive(bars + kSlotFull + s * 8);
        }
        if (++r == ring_entries) {
            r = 0;
            r_parity ^= 1;
        }
        if (++s == C::kSlots) {
            s = 0;
            s_parity ^= 1;
        }
    }
}

// ---------------------------------------------------------------------- MMA --
// Products come in turns n = 0, 1, ...: scores S(n) = Q K^T and outputs O += P(n) V.
// With two row tiles (pair) turns 2j and 2j + 1 are theirs for tile j of the keys; with
// one, turn n is tile n of the keys.  With two accumulators, turns of either parity have
// one each.  Barriers come in twos as well, one for each parity, whose phase n >> 1 is
// turn n's; only the one place for scores at head_dim 128 has a phase a turn.
//   S(n) goes where S(n - places) was: that has been read into registers by then (s_free)
//   P(n) goes where P(n - 2) was: its product has to be over (pv_done)
// Scores and outputs are issued by a warp each, so that scores run ahead of the softmax
// and neither's waits (70 cycles even where there is nothing to wait for; the tensor
// core takes in few products ahead) are in the other's way.
template <int D, int BITS>
struct Slots {
    using C = Cfg<D, BITS>;
    int entry = 0;
    uint32_t slot = 0, parity = 0;
    // Waits for entry e (entries are visited in order).
    __device__ __forceinline__ bool ready(const ChunkParams& p, int e, uint32_t bars) {
#pragma unroll 1
        for (; entry < e; ++entry)
            if (++slot == C::kSlots) {
                slot = 0;
                parity ^= 1;
            }
        return wait(p, bars, kSlotFull + slot * 8, parity);
    }
};

template <int D, int BITS>
__device__ __forceinline__ void scores_role(const ChunkParams& p, const Work& w, uint32_t q, uint32_t slots, uint32_t bars, bool pair) {
    using C = Cfg<D, BITS>;
    const uint32_t tmem = fixed(lds32(bars + kTmemAt)), q_op = fixed(smem_operand(q, 16)), k_op = fixed(smem_operand(slots, 16));
    const int turns = pair ? 2 * w.tiles : w.tiles;
    Slots<D, BITS> in;
    if (!wait(p, bars, kQFull, 0)) return;
#pragma unroll 1
    for (int n = 0; n < turns; ++n) {
        const bool first = !pair || (n & 1) == 0, last = !pair || (n & 1) != 0;
        if (first && !in.ready(p, key_entry(pair ? n >> 1 : n), bars)) return;
        if (n >= C::kPlaces) {
            const bool ok = C::kPlaces == 1 ? wait(p, bars, kSFree, (n - 1) & 1) : wait(p, bars, kSFree + (n & 1) * 8, ((n >> 1) - 1) & 1);
            if (!ok) return;
        }
        tc_fence_after();
        uint32_t a = q_op + (pair ? n & 1 : 0) * ((kRowTile * D * 2) >> 4), b = k_op + in.slot * (C::kSlot >> 4);
        const uint32_t s = tmem + (C::kPlaces == 2 ? (n & 1) * C::kS1 : 0);
        if (elect_one()) {
#pragma unroll 1
            for (int i = 0; i < D / 64; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_ss(s, a + k * 2, b + k * 2, mma_desc(kRowTile, C::kTile, false), k > 0 || i > 0);
                a += (kRowTile * 128) >> 4;
                b += (C::kTile * 128) >> 4;
            }
            tc_commit(bars + kSFull + (n & 1) * 8);
            if (last) tc_commit(bars + kSlotEmpty + in.slot * 8);
        }
        __syncwarp();
    }
}

template <int D, int BITS>
__device__ __forceinline__ void outputs_role(const ChunkParams& p, const Work& w, uint32_t slots, uint32_t bars, bool pair) {
    using C = Cfg<D, BITS>;
    const uint32_t tmem = fixed(lds32(bars + kTmemAt)), v_op = fixed(smem_operand(slots, C::kTile * 128));
    const int turns = pair ? 2 * w.tiles : w.tiles;
    Slots<D, BITS> in;
#pragma unroll 1
    for (int n = 0; n < turns; ++n) {
        const bool first = !pair || (n & 1) == 0, last = !pair || (n & 1) != 0;
        if (first && !in.ready(p, value_entry(pair ? n >> 1 : n, w.tiles), bars)) return;
        if (!wait(p, bars, kPFull + (n & 1) * 8, (n >> 1) & 1)) return;
        tc_fence_after();
        uint32_t b = v_op + in.slot * (C::kSlot >> 4), a = tmem + C::kP + (n & 1) * C::kPStep;
        const uint32_t o = tmem + C::kO + (C::kStreams == 2 ? (n & 1) * D : 0);
        const bool add = (n / C::kStreams & (C::kChain - 1)) != 0;  // (emptied accumulators begin anew)
        if (elect_one()) {
#pragma unroll 1
            for (int i = 0; i < C::kTile / 64; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_ts(o, a + k * 8, b + ((k * 2048) >> 4), mma_desc(kRowTile, D, true), k > 0 || i > 0 || add);
                a += 32;
                b += (4 * 2048) >> 4;
            }
            tc_commit(bars + kPvDone + (n & 1) * 8);
            if (last) tc_commit(bars + kSlotEmpty + in.slot * 8);
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ softmax --
// Position of channel c in the order of the operands (see unpack8).
template <int BITS>
__device__ __forceinline__ constexpr int place(int c) {
    return BITS == 4 ? (c & ~7) | ((c & 3) << 1) | ((c >> 2) & 1) : c;
}

// The 128 rows of a query tile from row tile_row0 of the item on, by 128 threads:
// 16 bytes a thread, rows behind the last as zeros.
template <int D, int BITS>
__device__ __forceinline__ void load_query(const ChunkParams& p, const Work& w, uint8_t* tile, int tid, int tile_row0) {
    constexpr int kPieces = D / 8;       // 16-byte pieces of a row: eight channels
    constexpr int kRows = 32 / kPieces;  // rows that a warp loads at a time
    constexpr int kAhead = 32 / kRows < 16 ? 32 / kRows : 16;
    const int lane = tid & 31, u = lane % kPieces, row0 = (tid >> 5) * 32;
    // lane l finds the warp's row l
    const int r = tile_row0 + row0 + lane;
    long long from = -1;
    if (r < w.rows) {
        int i, g;
        row_of(p, w.row0 + r, i, g);
        from = (w.h * p.group_q + g) * p.stride_h + i * p.stride_t;
    }
    const uint16_t* base = p.q + w.b * p.stride_b;
#pragma unroll 1
    for (int it0 = 0; it0 < 32 / kRows; it0 += kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int it = 0; it < kAhead; ++it) {
            const long long at = __shfl_sync(0xffffffffu, from, (it0 + it) * kRows + lane / kPieces);
            x[it] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(base + at) + u) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int it = 0; it < kAhead; ++it) {
            const int at = row0 + (it0 + it) * kRows + lane / kPieces;
            uint4 y = x[it];
            if (p.negate_q) y.x ^= 0x80008000u, y.y ^= 0x80008000u, y.z ^= 0x80008000u, y.w ^= 0x80008000u;
            if (BITS == 4)
                y = make_uint4(__byte_perm(y.x, y.z, 0x5410), __byte_perm(y.x, y.z, 0x7632), __byte_perm(y.y, y.w, 0x5410), __byte_perm(y.y, y.w, 0x7632));
            *reinterpret_cast<uint4*>(tile + (u / 8) * (kRowTile * 128) + at * 128 + (((u % 8) ^ (at & 7)) << 4)) = y;
        }
    }
}

// The same for a cache of rotated keys: a warp a row, turned in fp32 and rounded to fp16,
// the operand's type, once more.
template <int D, int BITS>
__device__ __forceinline__ void load_query_rotated(const ChunkParams& p, const Work& w, uint8_t* tile, int tid, int tile_row0) {
    constexpr int E = D / 32;
    const int lane = tid & 31;
    for (int at = tid >> 5; at < kRowTile; at += 4) {
        const int r = tile_row0 + at;
        float v[E] = {};
        if (r < w.rows) {
            int i, g;
            row_of(p, w.row0 + r, i, g);
            halves_to_floats<E>(p.q + w.b * p.stride_b + (w.h * p.group_q + g) * p.stride_h + i * p.stride_t + lane * E, v);
            hadamard_warp<E>(v, lane, p.rot_scale);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = lane * E + e, x = (c & ~63) | place<BITS>(c & 63);
            const __half q = __float2half_rn(p.negate_q ? -v[e] : v[e]);
            *reinterpret_cast<__half*>(tile + (x / 64) * (kRowTile * 128) + at * 128 + (((x / 8 % 8) ^ (at & 7)) << 4) + (x & 7) * 2) = q;
        }
    }
}

struct State {
    float m, l;  // what P counts from (log2 units: a maximum less kHead, -inf: none yet), sum
};

// Where a thread's row of an accumulator is emptied into: its sums as float4 [D / 4][128 rows],
// then what its weights count from and their sum, [2][128 rows].
template <int D, int BITS>
__device__ __forceinline__ float* chain_at(const ChunkParams& p, int stream) {
    return p.chains + (static_cast<long long>(blockIdx.x) * Cfg<D, BITS>::kStreams + stream) * (kRowTile * (D + 2));
}

// Empties an accumulator: its sums join those of the chains before.  A tensor core cuts
// sums off instead of rounding them: a step of 16 keys took 1.0e-7 off a sum of positive
// values (262,144 keys in one chain: 1.7e-3 of the output); a chain of 8,192 keys takes
// 5e-5, and chains are added in fp32 that rounds to nearest.  The sums count from where the
// first chain did, so that joining them reads nothing of them (loads in place of reductions,
// with the registers they take, made calls 5 to 12 % longer, this 0 to 3.5 %); weights that have
// grown by more than 2^64 start them anew (what they held is then below 2^-56 of the
// largest weight a key).
template <int D, int BITS>
__device__ __forceinline__ void empty_chain(const ChunkParams& p, uint32_t oa, int stream, bool first, State& st) {
    float* at = chain_at<D, BITS>(p, stream);
    float* own = at + kRowTile * D + (threadIdx.x & 127);
    const float up = first ? INFINITY : st.m - own[0];
    const bool anew = !(up <= 64.f);
    const float g = anew ? 1.f : ex2_approx(up);
    float4* sums = reinterpret_cast<float4*>(at) + (threadIdx.x & 127);
#pragma unroll 1
    for (int x = 0; x < D; x += 16, sums += 4 * kRowTile) {
        float o[16];
        tmem_ld16(oa + x, o);
        tmem_wait_ld();
        if (anew) {
#pragma unroll
            for (int y = 0; y < 4; ++y) sums[y * kRowTile] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) red_add4(sums + y * kRowTile, o[4 * y] * g, o[4 * y + 1] * g, o[4 * y + 2] * g, o[4 * y + 3] * g);
        }
    }
    if (anew) own[0] = st.m;
    own[kRowTile] = anew ? st.l : fmaf(st.l, g, own[kRowTile]);
    st.l = 0.f;
}

// The end of an accumulator that was emptied on its way: its sums come back into it.
template <int D, int BITS>
__device__ __forceinline__ void restore_chains(const ChunkParams& p, uint32_t oa, int stream, State& st) {
    __threadfence();  // the thread's own reductions are in what it reads
    const float* at = chain_at<D, BITS>(p, stream);
    const float* own = at + kRowTile * D + (threadIdx.x & 127);
    const float g = own[0] == -INFINITY ? 0.f : ex2_approx(own[0] - st.m);
    st.l = fmaf(own[kRowTile], g, st.l);
    const float4* sums = reinterpret_cast<const float4*>(at) + (threadIdx.x & 127);
#pragma unroll 1
    for (int x = 0; x < D; x += 16, sums += 4 * kRowTile) {
        float4 s[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) s[y] = __ldcg(sums + y * kRowTile);
        float o[16];
        tmem_ld16(oa + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = fmaf(reinterpret_cast<const float*>(s)[y], g, o[y]);
        tmem_st16(oa + x, reinterpret_cast<const uint32_t*>(o));
    }
    tmem_wait_st();
}

// One accumulator's turns: all, or (two accumulators) those of its parity; a thread a row.
template <int D, int BITS>
__device__ __forceinline__ bool softmax_loop(const ChunkParams& p, const Work& w, uint32_t bars, uint32_t tmem, int stream, bool pair, bool active, int lo, int hi, State& st) {
    using C = Cfg<D, BITS>;
    constexpr int N = C::kTile;
    const int lane = threadIdx.x & 31;
    const float c = p.score_scale_log2;
    const int turns = pair ? 2 * w.tiles : w.tiles;
#pragma unroll 1
    for (int n = stream; n < turns; n += C::kStreams) {
        const uint32_t odd = n & 1, phase = (n >> 1) & 1;
        if (!wait(p, bars, kSFull + odd * 8, phase)) return false;
        tc_fence_after();
        float s[N];
        if (active) {
            const uint32_t sa = tmem + (C::kPlaces == 2 ? odd * C::kS1 : 0);
#pragma unroll
            for (int x = 0; x < N; x += 32) tmem_ld32(sa + x, s + x);
        }
        if (active) tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(bars + kSFree + (C::kPlaces == 2 ? odd * 8 : 0));
        if (active) {
            const int t0 = (w.tile0 + (pair ? n >> 1 : n)) * N;
            if (__any_sync(0xffffffffu, t0 < lo || t0 + N > hi)) {
                const unsigned span = static_cast<unsigned>(hi > lo ? hi - lo : 0);
#pragma unroll
                for (int x = 0; x < N; ++x) s[x] = static_cast<unsigned>(t0 + x - lo) < span ? s[x] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < N; x += 2) mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], s[x], s[x + 1]);
            const float top = fmaf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), c, -kHead);
            const bool fresh = n < C::kStreams;                                             // nothing in O yet
            const bool begins = (n & (C::kChain * C::kStreams - 1)) < C::kStreams;          // a chain: the next product replaces O
            const bool grow = top > (fresh ? st.m : st.m + kLazy);
            if (begins || __any_sync(0xffffffffu, grow)) {
                const uint32_t oa = tmem + C::kO + (C::kStreams == 2 ? stream * D : 0);
                if (!fresh) {
                    // O holds the products of the turns before: all of them have to be over
                    const uint32_t before = C::kStreams == 1 ? n - 1 : n - 2;
                    if (!wait(p, bars, kPvDone + (before & 1) * 8, (before >> 1) & 1)) return false;
                    tc_fence_after();
                    if (begins) empty_chain<D, BITS>(p, oa, stream, n / C::kStreams == C::kChain, st);
                }
                const float f = grow ? ex2_approx(st.m - top) : 1.f;
                if (grow) st.m = top;
                st.l *= f;
                if (!begins) {
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        float o[16];
                        tmem_ld16(oa + x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] *= f;
                        tmem_st16(oa + x, reinterpret_cast<const uint32_t*>(o));
                    }
                }
            }
        }
        // P's columns are free once the product before the last is over
        if (n >= 2 && !wait(p, bars, kPvDone + odd * 8, phase ^ 1)) return false;
        if (active) {
            tc_fence_after();
            const float base = st.m == -INFINITY ? 0.f : -st.m;
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            const uint32_t pa = tmem + C::kP + odd * C::kPStep;
#pragma unroll
            for (int x = 0; x < N; x += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    float2 e = fma2(make_float2(s[x + 2 * y], s[x + 2 * y + 1]), make_float2(c, c), make_float2(base, base));
                    e.x = ex2_approx(e.x);
                    e.y = ex2_approx(e.y);
                    sum[y & 1] = add2(sum[y & 1], e);
                    pk[y] = pack_half2(e.x, e.y);
                }
                tmem_st16(pa + x / 2, pk);
            }
            sum[0] = add2(sum[0], sum[1]);
            st.l += sum[0].x + sum[0].y;
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(bars + kPFull + odd * 8);
    }
    return true;
}

template <int D, int BITS, bool ROT>
__device__ __forceinline__ void softmax_role(const ChunkParams& p, const Work& w, uint8_t* qs, uint8_t* slots, uint32_t bars, Bars* shared, int stream, bool pair) {
    using C = Cfg<D, BITS>;
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const int tile_row0 = pair ? stream * kRowTile : 0;
    const int r = tile_row0 + row;  // row of the item
    const bool valid = r < w.rows;
    const bool active = __any_sync(0xffffffffu, valid);
    if (pair || stream == 0) {
        uint8_t* tile = qs + (pair ? stream : 0) * (kRowTile * D * 2);
        if (ROT && p.rotate_q)
            load_query_rotated<D, BITS>(p, w, tile, row, tile_row0);
        else
            load_query<D, BITS>(p, w, tile, row, tile_row0);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) arrive(bars + kQFull);
    int i, g;
    row_of(p, w.row0 + (valid ? r : 0), i, g);
    // (rows behind the last are zeros that see everything: they ask for no masks)
    const int lo = valid ? first_key(p, i, w.ql, w.len) : 0, hi = valid ? end_key(p, i, w.ql, w.len) : 0x7fffffff;
    const uint32_t tmem = fixed(lds32(bars + kTmemAt) + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21));  // the warp's lanes
    State st{-INFINITY, 0.f};
    bool ok = softmax_loop<D, BITS>(p, w, bars, tmem, stream, pair, active, lo, hi, st);
    if (!ok) tmem_wait_st();  // given up: nothing is on its way to TMEM when it is freed
    // the last of this accumulator's products
    const int turns = pair ? 2 * w.tiles : w.tiles, last = C::kStreams == 1 ? turns - 1 : ((turns - 1 - stream) & ~1) + stream;
    if (ok && turns > stream) {
        ok = wait(p, bars, kPvDone + (last & 1) * 8, (last >> 1) & 1);
        tc_fence_after();
    }
    // Where both accumulators are those of one row tile, the second one's state through
    // shared memory (the operands' place: once all softmax threads are here no product
    // is left that reads them).
    const bool merge = !pair && C::kStreams == 2 && turns > 1;
    const uint32_t oa = tmem + C::kO + (C::kStreams == 2 ? stream * D : 0);
    if (ok && active && last >= C::kChain * C::kStreams) restore_chains<D, BITS>(p, oa, stream, st);
    float f = 1.f, fo = 0.f, m = st.m, l = st.l;
    asm volatile("barrier.cta.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
    float* apart = reinterpret_cast<float*>(qs);  // [D][129] of the second accumulator
    constexpr int kPad = kRowTile + 1;
    if (merge) {
        if (stream == 1 && ok && active) {
            shared->max[row] = st.m;
            shared->sum[row] = st.l;
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
                float o[16];
                tmem_ld16(oa + x, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) apart[(x + y) * kPad + row] = o[y];
            }
        }
        asm volatile("barrier.cta.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
        const float m1 = shared->max[row], l1 = shared->sum[row];
        m = fmaxf(st.m, m1);
        f = st.m == -INFINITY ? 0.f : ex2_approx(st.m - m);
        fo = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
        l = l * f + l1 * fo;
    }
    const bool mine = (pair || stream == 0) && ok && active;
    if (w.part < 0) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        f *= inv;
        fo *= inv;
    }
    // 32 columns of the output at a time
    auto columns = [&](int x, float (&v)[32]) {
        float o[32];
        if (turns > 0) {
            tmem_ld32(oa + x, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) {
            const int at = place<BITS>(y);
            v[y] = turns > 0 ? o[at] * f : 0.f;
            if (merge) v[y] += apart[(x + at) * kPad + row] * fo;
        }
    };
    if (!ROT || !p.rotate_out || w.part >= 0) {
        // Rows to shared memory (16 bytes apart from what would be the same banks), then
        // each to its place as one bulk copy: a thread's own stores, 16 bytes in each
        // of 32 rows at a time, took 10,000 cycles.
        const uint32_t stride = w.part >= 0 ? D * 4 + 16 : D * 2 + 16;
        uint8_t* to = (merge ? slots + C::kSlots * C::kSlot - kRowTile * (D * 4 + 16) : qs) + r * stride;
        if (mine) {
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float v[32];
                columns(x, v);
                if (w.part >= 0) {
#pragma unroll
                    for (int y = 0; y < 32; y += 4) *reinterpret_cast<float4*>(to + (x + y) * 4) = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                } else {
#pragma unroll
                    for (int y = 0; y < 32; y += 8) floats_to_halves<8>(*reinterpret_cast<float(*)[8]>(v + y), to + (x + y) * 2);
                }
            }
        }
        fence_proxy_async_shared();
        asm volatile("barrier.cta.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
        if (mine && valid) {
            const long long part = static_cast<long long>(w.part) * p.rows_per_item + r;
            void* dst = p.out + ((static_cast<long long>(w.b) * p.n + i) * p.num_q_heads + w.h * p.group_q + g) * D;
            if (w.part >= 0) {
                p.part_m[part] = m;
                p.part_l[part] = l;
                dst = p.part_acc + part * D;
            }
            bulk_store(dst, to, stride - 16);
            bulk_store_wait();
        }
        return;
    }
    // Values stored rotated: the rows through shared memory, then a warp a row.
    float* rows = reinterpret_cast<float*>(qs) + (pair ? stream : 0) * (D * kPad);
    if (mine) {
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
            float v[32];
            columns(x, v);
#pragma unroll
            for (int y = 0; y < 32; ++y) rows[(x + y) * kPad + row] = v[y];
        }
    }
    asm volatile("barrier.cta.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
    if (!ok || (!pair && stream == 1)) return;
    constexpr int E = D / 32;
    for (int at = row >> 5; at < kRowTile && tile_row0 + at < w.rows; at += 4) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = rows[(lane * E + e) * kPad + at];
        hadamard_warp<E>(v, lane, p.rot_scale);
        int ti, tg;
        row_of(p, w.row0 + tile_row0 + at, ti, tg);
        floats_to_halves<E>(v, p.out + ((static_cast<long long>(w.b) * p.n + ti) * p.num_q_heads + w.h * p.group_q + tg) * D + lane * E);
    }
}

// ------------------------------------------------------------------- kernel --
// ROT: with the transforms of rotated caches (apart, as they take registers and code).
template <int D, int BITS, bool ROT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<D, BITS>;
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    static_assert(offsetof(Bars, slot_empty) == kSlotEmpty && offsetof(Bars, s_full) == kSFull && offsetof(Bars, q_full) == kQFull && offsetof(Bars, abort) == kAbort, "addresses");
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);  // (an offset, so that it stays a shared-memory pointer)
    uint8_t* qs = base;
    uint8_t* slots = base + C::kQ;
    uint8_t* ring = slots + C::kSlots * C::kSlot;
    Work w;
    if (!find_work<C::kTile>(p, p.rows_per_item, w)) return;  // the whole CTA
    // (an item's rows may be fewer than its place has: one tile of them then)
    const bool pair = C::kStreams == 2 && w.rows > kRowTile;
    const int ring_entries = C::kRing + (pair ? 0 : C::kMoreRing);
    const int warp = threadIdx.x >> 5;
    if (warp == 16) {
        tmem_alloc(&bars.tmem, 512);
    } else if (warp == 17) {
        for (uint32_t at = (threadIdx.x & 31) * 8; at < kTmemAt; at += 32 * 8) {
            const bool by_unpack = at >= kRingEmpty && at < kSlotEmpty, by_softmax = (at >= kSFree && at < kSFree + 16) || (at >= kPFull && at < kPFull + 16);
            mbar_init(&bars.ring_full[0] + at / 8, by_unpack ? C::kUnpackWarps : (by_softmax ? 4 : (at == kQFull ? C::kStreams * 4 : 1)));
        }
        if (threadIdx.x == 17 * 32) bars.abort = 0;
        fence_mbarrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // registers: 640 x 96 at launch; 256 x 160 + 256 x 56 + 128 x 48 (one
    // accumulator: 128 x 160 + 128 x 24 + 256 x 56 + 128 x 48)
    if (warp < C::kSoftmax / 32) {
        regs_raise<160>();
        softmax_role<D, BITS, ROT>(p, w, qs, slots, fixed(smem_u32(&bars)), &bars, warp >> 2, pair);
    } else if (warp < 8) {
        regs_lower<24>();
    } else if (warp < 16) {
        regs_lower<56>();
        unpack_role<D, BITS>(p, w, fixed(smem_u32(ring)), fixed(smem_u32(qs + kRowTile * D * 2)), ring_entries, fixed(smem_u32(slots)), fixed(smem_u32(&bars)));
    } else {
        regs_lower<48>();
        if (warp == 16 || warp == 18) {
            const uint32_t at = fixed(smem_u32(&bars)), in = fixed(smem_u32(slots));
            if (warp == 16)
                scores_role<D, BITS>(p, w, fixed(smem_u32(qs)), in, at, pair);
            else
                outputs_role<D, BITS>(p, w, in, at, pair);
            __syncwarp();
            // products in flight end before the CTA leaves (they may be where a warp has given up)
            const uint32_t bar = at + kDrain + (warp == 18 ? 8 : 0);
            if (elect_one()) tc_commit(bar);
            __syncwarp();
            for (int it = 0; it < 1 << 20 && !over(bar, 0); ++it) {
            }
        } else if (warp == 17) {
            load_role<D, BITS>(p, w, fixed(smem_u32(ring)), fixed(smem_u32(qs + kRowTile * D * 2)), ring_entries, fixed(smem_u32(&bars)));
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_free(bars.tmem, 512);
    }
}

// -------------------------------------------------------------------- merge --
// A warp a row: the weights 2^(m_s - M) of the parts, then their sums.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(ChunkParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    pdl_wait_primary();
    const long long wid = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
    // row r of the item-th split item
    const int item = static_cast<int>(wid / p.rows_per_item), r = static_cast<int>(wid - static_cast<long long>(item) * p.rows_per_item);
    const int id = p.whole + item, all = p.batch * p.num_kv_heads;
    if (id >= all * p.m_items) return;
    const int above = id / all, bh = id - above * all, b = bh / p.num_kv_heads, h = bh - b * p.num_kv_heads;
    const int flat = (p.m_items - 1 - above) * p.rows_per_item + r;
    int i, g;
    row_of(p, flat, i, g);
    const int ql = p.q_lens != nullptr ? min(max(p.q_lens[b], 0), p.n) : p.n;
    if (i >= ql) return;
    const long long part0 = static_cast<long long>(item) * p.n_splits;
    float top = -INFINITY;
    for (int s = lane; s < p.n_splits; s += 32) top = fmaxf(top, p.part_m[(part0 + s) * p.rows_per_item + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[E] = {}, l = 0.f;
    const float* from = p.part_acc + (part0 * p.rows_per_item + r) * D + lane * E;
    const long long step = static_cast<long long>(p.rows_per_item) * D;
    for (int s0 = 0; s0 < p.n_splits; s0 += 32) {
        float f = 0.f, pl = 0.f;
        if (s0 + lane < p.n_splits) {
            const long long at = (part0 + s0 + lane) * p.rows_per_item + r;
            const float pm = p.part_m[at];
            f = pm == -INFINITY ? 0.f : ex2_approx(pm - top);
            pl = f * p.part_l[at];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pl += __shfl_xor_sync(0xffffffffu, pl, o);
        l += pl;
        // four parts' loads at a time (a part without a key in sight holds zeros)
        const int n = min(32, p.n_splits - s0);
        for (int s = 0; s < n; s += 4) {
            float v[4][E];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (s + k < n) {
                    if (E == 2)
                        *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(from + (s0 + s + k) * step);
                    else
#pragma unroll
                        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(v[k] + e) = *reinterpret_cast<const float4*>(from + (s0 + s + k) * step + e);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float fs = __shfl_sync(0xffffffffu, f, (s + k) & 31);
                if (s + k < n) {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(fs, v[k][e], acc[e]);
                }
            }
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    if (p.rotate_out) hadamard_warp<E>(acc, lane, p.rot_scale);
    uint16_t* out = p.out + ((static_cast<long long>(b) * p.n + i) * p.num_q_heads + h * p.group_q + g) * D + lane * E;
    floats_to_halves<E>(acc, out);
}

template <int D, int BITS, bool ROT>
cudaError_t launch_main(const ChunkParams& p, cudaStream_t stream) {
    using C = Cfg<D, BITS>;
    cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, BITS, ROT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const long long ctas = p.whole + (static_cast<long long>(p.batch) * p.num_kv_heads * p.m_items - p.whole) * p.n_splits;
    chunk_kernel<D, BITS, ROT><<<static_cast<unsigned>(ctas), kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const ChunkParams& p, cudaStream_t stream) {
    const bool rot = p.rotate_q || (p.rotate_out && (p.n_splits == 1 || p.whole > 0));
    cudaError_t e = p.bits == 8 ? (rot ? launch_main<D, 8, true>(p, stream) : launch_main<D, 8, false>(p, stream))
                                : (rot ? launch_main<D, 4, true>(p, stream) : launch_main<D, 4, false>(p, stream));
    if (e != cudaSuccess || p.n_splits == 1) return e;
    const long long rows = (static_cast<long long>(p.batch) * p.num_kv_heads * p.m_items - p.whole) * p.rows_per_item, each = kMergeThreads / 32;
    return launch_after(chunk_merge_kernel<D>, static_cast<unsigned>((rows + each - 1) / each), kMergeThreads, stream, p);
}

}  // namespace

int chunk_tile_tokens(int head_dim) { return head_dim == 256 ? Cfg<256, 4>::kTile : Cfg<128, 4>::kTile; }

size_t chunk_chain_floats(int head_dim) { return static_cast<size_t>(head_dim == 256 ? Cfg<256, 4>::kStreams : Cfg<128, 4>::kStreams) * kRowTile * (head_dim + 2); }

cudaError_t launch_chunk(const ChunkParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch_dim<64>(p, stream);
    return head_dim == 128 ? launch_dim<128>(p, stream) : launch_dim<256>(p, stream);
}

}  // namespace tq
