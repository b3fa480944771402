// chunk.cu -- attention of several query rows per sequence over the cache: a
// chunk of new tokens in causal order (optionally the last `window` tokens
// only), or every row over the whole sequence.  For row r = (token i, head g) of
// (sequence b, kv head h), r = i * G + g:
//   out_r = sum_t p_t V_t / sum_t p_t,  p_t = 2^(c q_r.K_t - m_r),  lo_i <= t < hi_i,
// with c = attn_scale log2(e) and m_r a running maximum.  Rows of all the heads
// that share a kv head are rows of one matrix, so every cached key and value is
// unpacked once for 256 of them.
//
// A CTA takes 256 rows (two tiles of 128, the M of a tcgen05.mma; one tile at
// head_dim 256, whose output fills half of TMEM) and a run of the keys they see, in
// tiles of 128 (64 at head_dim 256):
//   a loader thread   copies codes, scales and biases into a ring (bulk copies)
//   unpacking warps   turn them into fp16 operands in shared memory, laid out as
//                     128-byte rows with the 128-byte swizzle: keys are then a
//                     K-major operand and values an N-major one, in the same layout
//   MMA warps         S = Q K^T and O += P V, S, P and O in TMEM (P in S's place)
//   softmax warps     a thread a row: maximum, 2^x, P as fp16, sum; no shuffles
// The two row tiles take turns: while one's softmax runs the tensor core works for
// the other.  Up to 128 rows (a few tokens) make one tile; the two halves then take
// every other tile of keys and are merged in the end.  O is rescaled only when a
// row's maximum grows by more than 2^8 (P stays below 2^8, exact enough in fp16's
// range; the method of the published conditional-rescaling softmax), which is
// rare after the first tiles.
// Where rows are few the keys are split over CTAs and the partial states
// merged by a second kernel.
#include <stddef.h>

#include "tq_device.cuh"
#include "tq_hadamard.cuh"
#include "tq_internal.h"
#include "tq_tcgen05.cuh"

namespace tq {

namespace {

constexpr int kThreads = 640;       // 8 softmax warps, 8 that unpack, 2 that issue products, one that copies
constexpr int kRowTile = 128;
constexpr float kLazy = 8.f;  // log2 of how far P may grow before O is rescaled

template <int D, int BITS>
struct Cfg {
    static constexpr int kStreams = D == 256 ? 1 : 2;         // softmax warpgroups, output accumulators
    static constexpr int kTile = D == 256 ? 64 : 128;         // keys
    static constexpr int kUnpackWarp = 8;                     // first unpacking warp
    static constexpr int kUnpackWarps = 8;
    static constexpr int kBlocks = D / 64;                    // blocks of 64 channels: 128-byte rows
    static constexpr int kSlot = kTile * D * 2;               // one unpacked tile of keys or values
    static constexpr int kSlots = D == 64 ? 6 : 3;
    static constexpr int kCodes = kTile * D * BITS / 8;
    static constexpr int kScales = kTile * kBlocks * 2;       // scales (and as many biases) of a tile
    static constexpr int kEntry = kCodes + 2 * kScales;
    static constexpr int kRing = D == 64 ? 6 : (BITS == 8 ? 3 : 6);
    static constexpr int kQ = kStreams * kRowTile * D * 2;
    static constexpr int kSmem = 1024 + kQ + kSlots * kSlot + kRing * kEntry;
    static constexpr uint32_t kS = kTile;                     // TMEM columns of S; P lies in their upper half
    static constexpr uint32_t kO = 256;                       // first TMEM column of O
    static_assert(kSmem + 512 <= 232448, "shared memory of a CTA");
    static_assert(kO + kStreams * D <= 512 && 2 * kS <= kO, "TMEM");
};

struct Bars {
    uint64_t ring_full[6], ring_empty[6], slot_full[6], slot_empty[6];
    uint64_t s_full[2], p_full[2], o_full[2], q_full, drain[2], half;
    uint32_t tmem;
    int32_t abort;
};

// Addresses of the barriers from that of the first.  (Each role takes the first one's
// once, in a way that the compiler cannot repeat: left to it, it forms a shared
// variable's address anew wherever it is used, from a special register that takes
// tens of cycles to read, which between two products is time lost.)
enum : uint32_t {
    kRingFull = 0,
    kRingEmpty = 6 * 8,
    kSlotFull = 12 * 8,
    kSlotEmpty = 18 * 8,
    kSFull = 24 * 8,
    kPFull = 26 * 8,
    kOFull = 28 * 8,
    kQFull = 30 * 8,
    kDrain = 31 * 8,
    kHalf = 33 * 8,
    kTmemAt = 34 * 8,
    kAbort = 34 * 8 + 4,
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

// What a CTA works on.
struct Work {
    int b, h, part;         // part: (item, split), where partial states go
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
    // the last rows' items first: in causal order they see the most keys
    int id = blockIdx.x;
    const int per = p.batch * p.num_kv_heads * p.n_splits;
    const int m = p.m_items - 1 - id / per;
    id %= per;
    const int split = id % p.n_splits;
    const int bh = id / p.n_splits;
    w.h = bh % p.num_kv_heads;
    w.b = bh / p.num_kv_heads;
    w.part = (bh * p.m_items + m) * p.n_splits + split;
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
    w.klo = first_key(p, w.row0 / p.group_q, ql, len);
    w.khi = end_key(p, (w.row0 + w.rows - 1) / p.group_q, ql, len);
    w.tile0 = w.klo / TILE;
    const int all = w.khi > w.klo ? (w.khi + TILE - 1) / TILE - w.tile0 : 0;
    const int t0 = static_cast<int>(static_cast<long long>(all) * split / p.n_splits);
    w.tiles = static_cast<int>(static_cast<long long>(all) * (split + 1) / p.n_splits) - t0;
    w.tile0 += t0;
    return true;
}

// Entry e of the ring holds the keys or the values of tile `tile`.  pair: both row
// tiles use a tile of keys, then its values (K0 V0 K1 V1 ...); else the next
// keys come ahead of the values (K0 K1 V0 K2 V1 ... V_last).
__device__ __forceinline__ bool entry_of(int e, int tiles, bool pair, int& tile) {
    if (pair) {
        tile = e >> 1;
        return (e & 1) != 0;
    }
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
__device__ __forceinline__ int key_entry(int tile, bool pair) { return pair ? 2 * tile : (tile == 0 ? 0 : 2 * tile - 1); }
__device__ __forceinline__ int value_entry(int tile, int tiles, bool pair) {
    return pair ? 2 * tile + 1 : (tile == tiles - 1 ? 2 * tiles - 1 : 2 * tile + 2);
}

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

// Waits for a phase of the barrier at `bar`; false when it took too long or another
// warp has given up.  (The timer is read rarely: that takes longer than most waits.)
__device__ __forceinline__ bool wait(uint32_t bars, uint32_t bar, uint32_t parity, int32_t* status) {
    if (over(bars + bar, parity)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (over(bars + bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (lds32(bars + kAbort) != 0) return false;
            const uint64_t now = (it & 1023u) == 0 ? globaltimer_ns() : 0;
            if (now != 0 && t0 == 0) t0 = now;
            if (now != 0 && now - t0 > 2000000000ull) {
                asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(bars + kAbort) : "memory");
                if (status != nullptr) atomicOr(status, TQ_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

// ------------------------------------------------------------------ loader --
template <int D, int BITS>
__device__ __forceinline__ void load_role(const ChunkParams& p, const Work& w, uint8_t* ring, Bars* bars, bool pair) {
    using C = Cfg<D, BITS>;
    const uint64_t policy = policy_evict_first();
    const uint32_t at = fixed(smem_u32(bars));
    int e = 0;
#pragma unroll 1
    for (; e < 2 * w.tiles; ++e) {
        const int r = e % C::kRing, n = e / C::kRing;
        if (n > 0 && !wait(at, kRingEmpty + r * 8, (n - 1) & 1, p.status)) break;
        int tile;
        const bool value = entry_of(e, w.tiles, pair, tile);
        const int t0 = (w.tile0 + tile) * C::kTile;
        const int rows = min(C::kTile, (w.khi - t0 + 15) & ~15);  // capacities are whole 16s
        const long long row = kv_row(p.map, p.num_kv_heads, w.b, w.h, t0, p.status);
        uint8_t* dst = ring + r * C::kEntry;
        const uint32_t cb = rows * (D * BITS / 8), sb = rows * (C::kBlocks * 2);
        mbar_arrive_expect_tx(&bars->ring_full[r], cb + 2 * sb);
        bulk_load(dst, (value ? p.v_codes : p.k_codes) + row * (D * BITS / 8), cb, &bars->ring_full[r], policy);
        bulk_load(dst + C::kCodes, (value ? p.v_scale : p.k_scale) + row * C::kBlocks, sb, &bars->ring_full[r], policy);
        bulk_load(dst + C::kCodes + C::kScales, (value ? p.v_bias : p.k_bias) + row * C::kBlocks, sb, &bars->ring_full[r], policy);
    }
    if (e < 2 * w.tiles)  // given up: the copies in flight land before the CTA leaves
        for (int k = max(0, e - C::kRing); k < e; ++k) mbar_wait_bounded(&bars->ring_full[k % C::kRing], (k / C::kRing) & 1);
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
__device__ __forceinline__ void unpack_role(const ChunkParams& p, const Work& w, uint32_t ring, uint32_t slots, uint32_t bars, bool pair) {
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
    const uint32_t from = ring + tid * 16, from_scale = ring + C::kCodes + (t * C::kBlocks + g) * 2;
    int r = 0, s = 0;
    uint32_t r_parity = 0, s_parity = 1;
#pragma unroll 1
    for (int e = 0; e < 2 * w.tiles; ++e) {
        if (!wait(bars, kRingFull + r * 8, r_parity, p.status)) return;
        if (!wait(bars, kSlotEmpty + s * 8, s_parity, p.status)) return;  // (a fresh barrier's phase before the first is over)
        int tile;
        const bool value = entry_of(e, w.tiles, pair, tile);
        const int t0 = (w.tile0 + tile) * C::kTile;
        const uint32_t src = from + r * C::kEntry, src_scale = from_scale + r * C::kEntry, dst = s * C::kSlot;
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
        if (++r == C::kRing) {
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
// Run by whole warps, an elected lane of which issues.  The tensor core takes in few
// products ahead, so what is between two of them (waits of 70 cycles even when there
// is nothing to wait for, commits of 50) is time that it stands still: with two
// accumulators a warp for each issues, one's products filling the other's gaps.
template <int D, int BITS>
struct Products {
    using C = Cfg<D, BITS>;
    uint32_t bars, tmem, q_op, k_op, v_op;
    int32_t* status;
    // the slot that an entry is in: entries are visited in order, some left out
    int entry;
    uint32_t slot, parity;
    __device__ __forceinline__ bool ready(int e) {
#pragma unroll 1
        for (; entry < e; ++entry)
            if (++slot == C::kSlots) {
                slot = 0;
                parity ^= 1;
            }
        const bool ok = wait(bars, kSlotFull + slot * 8, parity, status);
        tc_fence_after();
        return ok;
    }
    // S[buf] = Q[qt] K^T, the keys in the current slot
    __device__ __forceinline__ void scores(uint32_t qt, uint32_t buf) const {
        uint32_t a = q_op + qt * ((kRowTile * D * 2) >> 4), b = k_op + slot * (C::kSlot >> 4);
        const uint32_t s = tmem + buf * C::kS;
        if (elect_one()) {
#pragma unroll 1
            for (int i = 0; i < D / 64; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_ss(s, a + k * 2, b + k * 2, mma_desc(kRowTile, C::kTile, false), k > 0 || i > 0);
                a += (kRowTile * 128) >> 4;
                b += (C::kTile * 128) >> 4;
            }
            tc_commit(bars + kSFull + buf * 8);
            tc_commit(bars + kSlotEmpty + slot * 8);
        }
        __syncwarp();
    }
    // O[o] (+)= P[buf] V, the values in the current slot
    __device__ __forceinline__ void outputs(uint32_t buf, uint32_t o, bool add, bool told) const {
        uint32_t b = v_op + slot * (C::kSlot >> 4), s = tmem + buf * C::kS + C::kS / 2;
        const uint32_t d = tmem + C::kO + o * D;
        if (elect_one()) {
#pragma unroll 1
            for (int i = 0; i < C::kTile / 64; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_ts(d, s + k * 8, b + ((k * 2048) >> 4), mma_desc(kRowTile, D, true), k > 0 || i > 0 || add);
                s += 32;
                b += (4 * 2048) >> 4;
            }
            tc_commit(bars + kSlotEmpty + slot * 8);
            if (told) tc_commit(bars + kOFull + o * 8);
        }
        __syncwarp();
    }
};

// The tiles of one accumulator: all (pair) or every other one.
template <int D, int BITS>
__device__ __forceinline__ bool mma_loop(const ChunkParams& p, const Work& w, uint32_t q, uint32_t slots, uint32_t bars, bool pair, uint32_t stream) {
    using C = Cfg<D, BITS>;
    Products<D, BITS> x{bars, fixed(lds32(bars + kTmemAt)), fixed(smem_operand(q, 16)), fixed(smem_operand(slots, 16)), fixed(smem_operand(slots, C::kTile * 128)),
                        p.status, 0, 0, 0};
    if (!wait(bars, kQFull, 0, p.status)) return false;
    const int T = w.tiles;
    if (C::kStreams == 2) {
        const int step = pair ? 1 : 2;
        const uint32_t qt = pair ? stream : 0;
        int j = pair ? 0 : stream;
        if (j >= T) return true;
        // the second row tile half a turn behind the first: in step, both would wait for
        // their softmax at the same time
        if (pair && stream == 1 && !wait(bars, kHalf, 0, p.status)) return false;
        if (!x.ready(key_entry(j, pair))) return false;
        tc_fence_after();
        x.scores(qt, stream);
#pragma unroll 1
        for (uint32_t k = 0; j < T; ++k, j += step) {
            if (!x.ready(value_entry(j, T, pair)) || !wait(bars, kPFull + stream * 8, k & 1, p.status)) return false;
            tc_fence_after();
            x.outputs(stream, stream, k > 0, j + step >= T);
            if (j + step < T) {
                if (!x.ready(key_entry(j + step, pair))) return false;
                x.scores(qt, stream);
            }
        }
        return true;
    }
    // one accumulator, two places for scores
    for (int j = 0; j < 2 && j < T; ++j) {
        if (!x.ready(key_entry(j, false))) return false;
        tc_fence_after();
        x.scores(0, j);
    }
#pragma unroll 1
    for (int j = 0; j < T; ++j) {
        if (!x.ready(value_entry(j, T, false)) || !wait(bars, kPFull + (j & 1) * 8, (j >> 1) & 1, p.status)) return false;
        tc_fence_after();
        x.outputs(j & 1, 0, j > 0, true);  // (told of every one: the softmax may have to rescale the sums before the next)
        if (j + 2 < T) {
            if (!x.ready(key_entry(j + 2, false))) return false;
            x.scores(0, j & 1);
        }
    }
    return true;
}

// ------------------------------------------------------------------ softmax --
// Position of channel c in the order of the operands (see unpack8).
template <int BITS>
__device__ __forceinline__ constexpr int place(int c) {
    return BITS == 4 ? (c & ~7) | ((c & 3) << 1) | ((c >> 2) & 1) : c;
}

// The fast transform of N values in one thread's registers.
template <int N>
__device__ __forceinline__ void hadamard_thread(float (&v)[N]) {
#pragma unroll
    for (int h = 1; h < N; h <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if ((i & h) == 0) {
                const float u = v[i], x = v[i + h];
                v[i] = u + x;
                v[i + h] = u - x;
            }
        }
    }
}

// 64 channels (a 128-byte row of one block) of row `row` of a query tile.
template <int BITS>
__device__ __forceinline__ void store_q64(uint8_t* block, int row, const __half2 (&x)[32]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint4 o;
        uint32_t* w = reinterpret_cast<uint32_t*>(&o);
        const uint32_t* s = reinterpret_cast<const uint32_t*>(x) + u * 4;
        if (BITS == 4) {
            w[0] = __byte_perm(s[0], s[2], 0x5410);
            w[1] = __byte_perm(s[0], s[2], 0x7632);
            w[2] = __byte_perm(s[1], s[3], 0x5410);
            w[3] = __byte_perm(s[1], s[3], 0x7632);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = s[k];
        }
        *reinterpret_cast<uint4*>(block + row * 128 + ((u ^ (row & 7)) << 4)) = o;
    }
}

// The 128 rows of a query tile from row tile_row0 of the item on, by one warpgroup
// (thread `row`): 16 bytes a thread, rows behind the last as zeros.
template <int D, int BITS>
__device__ __forceinline__ void load_query(const ChunkParams& p, const Work& w, uint8_t* tile, int row, int tile_row0) {
    constexpr int kPieces = D / 8;  // 16-byte pieces of a row: eight channels
    const int u = row % kPieces;
#pragma unroll 8
    for (int it = 0; it < kPieces; ++it) {
        const int at = it * (128 / kPieces) + row / kPieces, r = tile_row0 + at;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < w.rows) {
            const int flat = w.row0 + r, i = flat / p.group_q, g = flat - i * p.group_q;
            x = __ldg(reinterpret_cast<const uint4*>(p.q + w.b * p.stride_b + (w.h * p.group_q + g) * p.stride_h + i * p.stride_t) + u);
        }
        if (p.negate_q) x.x ^= 0x80008000u, x.y ^= 0x80008000u, x.z ^= 0x80008000u, x.w ^= 0x80008000u;
        if (BITS == 4)
            x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
        *reinterpret_cast<uint4*>(tile + (u / 8) * (kRowTile * 128) + at * 128 + (((u % 8) ^ (at & 7)) << 4)) = x;
    }
}

// The same for a cache of rotated keys: a thread a row.
template <int D, int BITS>
__device__ __forceinline__ void load_query_rotated(const ChunkParams& p, const Work& w, uint8_t* tile, int row, int tile_row0) {
    const int r = tile_row0 + row;
    const bool valid = r < w.rows;
    const int flat = w.row0 + (valid ? r : 0), i = flat / p.group_q, g = flat - i * p.group_q;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + w.b * p.stride_b + (w.h * p.group_q + g) * p.stride_h + i * p.stride_t);
    constexpr int N = D < 128 ? D : 128;
    for (int half = 0; half < D / N; ++half) {
        float v[N];
#pragma unroll
        for (int u = 0; u < N / 8; ++u) {
            uint4 x = valid ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
            halves_to_floats<8>(&x, *reinterpret_cast<float(*)[8]>(v + u * 8));
            if (D == 256) {  // the stage of 128 first: sums for the first half, differences for the second
                float y[8];
                x = valid ? __ldg(src + 16 + u) : make_uint4(0, 0, 0, 0);
                halves_to_floats<8>(&x, y);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[u * 8 + k] = half ? v[u * 8 + k] - y[k] : v[u * 8 + k] + y[k];
            }
        }
        hadamard_thread<N>(v);
        const float scale = p.negate_q ? -p.rot_scale : p.rot_scale;
#pragma unroll
        for (int blk = 0; blk < N / 64; ++blk) {
            __half2 x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __floats2half2_rn(v[blk * 64 + 2 * k] * scale, v[blk * 64 + 2 * k + 1] * scale);
            store_q64<BITS>(tile + (half * (N / 64) + blk) * (kRowTile * 128), row, x);
        }
    }
}

struct State {
    float m, l;  // maximum that P counts from (log2 units, -inf: none yet), sum
};

// One warpgroup's tiles: j = first, first + step, ...
template <int D, int BITS>
__device__ __forceinline__ bool softmax_loop(const ChunkParams& p, const Work& w, uint32_t bars, uint32_t tmem0, int stream, bool pair, bool active, int lo, int hi, State& st) {
    using C = Cfg<D, BITS>;
    constexpr int N = C::kTile;
    const int lane = threadIdx.x & 31;
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
    const uint32_t tmem = tmem0 + lanes;
    const float c = p.score_scale_log2;
    const int step = pair || C::kStreams == 1 ? 1 : 2;
    for (int j = step == 2 ? stream : 0, k = 0; j < w.tiles; j += step, ++k) {
        const int buf = pair || C::kStreams == 2 ? stream : j & 1;
        const uint32_t phase = C::kStreams == 1 ? (j >> 1) & 1 : k & 1;
        if (!wait(bars, kSFull + buf * 8, phase, p.status)) return false;
        tc_fence_after();
        if (active) {
            const uint32_t sa = tmem + buf * C::kS;
            const int t0 = (w.tile0 + j) * C::kTile;
            if (__any_sync(0xffffffffu, t0 < lo || t0 + N > hi)) {
                // scores of keys that the row does not see: minus infinity, once and for both passes
                const unsigned span = static_cast<unsigned>(hi > lo ? hi - lo : 0);
#pragma unroll 1
                for (int x = 0; x < N; x += 32) {
                    float s[32];
                    tmem_ld32(sa + x, s);
                    tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 32; ++y) s[y] = static_cast<unsigned>(t0 + x + y - lo) < span ? s[y] : -INFINITY;
                    tmem_st32(sa + x, s);
                }
                tmem_wait_st();
            }
            // Two passes over the scores in TMEM, 32 columns at a time with the next 32 on
            // their way, in loops (unrolled, the code of the roles that share an
            // instruction cache did not fit it: products were issued at half the rate).
            float u[32], v[32];
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto highest = [&mx](const float (&s)[32]) {
#pragma unroll
                for (int x = 0; x < 32; x += 2) mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], s[x], s[x + 1]);
            };
            tmem_ld32(sa, u);
#pragma unroll 1
            for (int x = 0; x < N; x += 64) {
                tmem_wait_ld();
                tmem_ld32(sa + x + 32, v);
                highest(u);
                tmem_wait_ld();
                tmem_ld32(sa + (x + 64) % N, u);
                highest(v);
            }
            tmem_wait_ld();
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
            const bool grow = k == 0 ? top > st.m : top > st.m + kLazy;
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2_approx(st.m - top) : 1.f;
                if (grow) st.m = top;
                st.l *= f;
                if (k > 0) {
                    // O holds the products up to the tile before; with one accumulator the
                    // last of them may still run (with two, this S came after it)
                    if (C::kStreams == 1) {
                        if (!wait(bars, kOFull, (j - 1) & 1, p.status)) return false;
                        tc_fence_after();
                    }
                    const uint32_t oa = tmem + C::kO + (C::kStreams == 2 ? stream * D : 0);
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        float o[32];
                        tmem_ld32(oa + x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] *= f;
                        tmem_st32(oa + x, o);
                    }
                }
            }
            const float base = st.m == -INFINITY ? 0.f : -st.m;
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            // from the last column down: P's columns are those of scores already read
            auto weights = [&](const float (&s)[32], int x) {
                uint32_t pk[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    float2 e = fma2(make_float2(s[2 * y], s[2 * y + 1]), make_float2(c, c), make_float2(base, base));
                    e.x = ex2_approx(e.x);
                    e.y = ex2_approx(e.y);
                    sum[y & 1] = add2(sum[y & 1], e);
                    pk[y] = pack_half2(e.x, e.y);
                }
                tmem_st16(sa + C::kS / 2 + x / 2, pk);
            };
            tmem_ld32(sa + N - 32, u);
#pragma unroll 1
            for (int x = N - 32; x > 0; x -= 64) {
                tmem_wait_ld();
                tmem_ld32(sa + x - 32, v);
                weights(u, x);
                tmem_wait_ld();
                if (x > 64) tmem_ld32(sa + x - 64, u);
                weights(v, x - 32);
            }
            sum[0] = add2(sum[0], sum[1]);
            st.l += sum[0].x + sum[0].y;
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            arrive(bars + kPFull + buf * 8);
            if (C::kStreams == 2 && stream == 0 && k == 0) arrive(bars + kHalf);
        }
    }
    return true;
}

// The output row of one thread, from TMEM (merge: + other's columns in shared memory).
template <int D, int BITS, bool ROT>
__device__ __forceinline__ void write_row(const ChunkParams& p, const Work& w, uint32_t oa, bool has, bool valid, int r, const State& st, float f,
                                          const float* other, float fo) {
    const int flat = w.row0 + r, i = flat / p.group_q, g = flat - i * p.group_q;
    // 32 columns of O, scaled, by channel
    auto columns = [&](int x, float (&v)[32]) {
        float o[32];
        if (has) {
            tmem_ld32(oa + x, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) {
            const int at = place<BITS>(y);
            v[y] = has ? o[at] * f : 0.f;
            if (other != nullptr) v[y] += other[(x + at) * kRowTile] * fo;
        }
    };
    if (p.n_splits > 1) {
        const long long at = static_cast<long long>(w.part) * p.rows_per_item + r;
        if (valid) {
            p.part_m[at] = st.m;
            p.part_l[at] = st.l;
        }
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
            float v[32];
            columns(x, v);
            if (valid) {
#pragma unroll
                for (int y = 0; y < 32; y += 4)
                    *reinterpret_cast<float4*>(p.part_acc + at * D + x + y) = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
            }
        }
        return;
    }
    uint16_t* out = p.out + ((static_cast<long long>(w.b) * p.n + i) * p.num_q_heads + w.h * p.group_q + g) * D;
    if (!ROT || !p.rotate_out) {
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
            float v[32];
            columns(x, v);
            if (valid) {
#pragma unroll
                for (int y = 0; y < 32; y += 8) {
                    uint4 o;
                    floats_to_halves<8>(*reinterpret_cast<float(*)[8]>(v + y), &o);
                    *reinterpret_cast<uint4*>(out + x + y) = o;
                }
            }
        }
        return;
    }
    constexpr int N = D < 128 ? D : 128;
    for (int half = 0; half < D / N; ++half) {
        float v[N];
#pragma unroll
        for (int x = 0; x < N; x += 32) {
            columns(x, *reinterpret_cast<float(*)[32]>(v + x));
            if (D == 256) {
                float y[32];
                columns(128 + x, y);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[x + k] = half ? v[x + k] - y[k] : v[x + k] + y[k];
            }
        }
        hadamard_thread<N>(v);
        if (valid) {
#pragma unroll
            for (int y = 0; y < N; y += 8) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = v[y + k] * p.rot_scale;
                uint4 o;
                floats_to_halves<8>(x, &o);
                *reinterpret_cast<uint4*>(out + half * N + y) = o;
            }
        }
    }
}

template <int D, int BITS, bool ROT>
__device__ __forceinline__ void softmax_role(const ChunkParams& p, const Work& w, uint8_t* qs, uint8_t* slots, uint32_t bars, int stream, bool pair) {
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
    const int i = (w.row0 + (valid ? r : 0)) / p.group_q;
    // (rows behind the last are zeros that see everything: they ask for no masks)
    const int lo = valid ? first_key(p, i, w.ql, w.len) : 0, hi = valid ? end_key(p, i, w.ql, w.len) : 0x7fffffff;
    const uint32_t tmem = fixed(lds32(bars + kTmemAt));
    State st{-INFINITY, 0.f};
    const bool done = softmax_loop<D, BITS>(p, w, bars, tmem, stream, pair, active, lo, hi, st);
    const bool split_keys = !pair && C::kStreams == 2;
    // tiles of this stream, and the phase of its accumulator's last barrier
    const int mine = split_keys ? (w.tiles + 1 - stream) / 2 : w.tiles;
    bool ok = done;
    if (ok && mine > 0) {
        // (one accumulator: a phase a tile, of which the last score tile shows all but the last two to be over)
        if (C::kStreams == 1 && mine > 1) ok = wait(bars, kOFull, (mine - 2) & 1, p.status);
        ok = ok && wait(bars, kOFull + (C::kStreams == 2 ? stream : 0) * 8, C::kStreams == 1 ? (mine - 1) & 1 : 0, p.status);
        tc_fence_after();
    }
    const uint32_t oa = tmem + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21) + C::kO + (C::kStreams == 2 ? stream * D : 0);
    if (split_keys) {
        // the second half's state through shared memory (the operands' place: no product is left that reads them)
        float* buf = reinterpret_cast<float*>(slots);  // [D][128], then m and l
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (stream == 1 && ok && active) {
#pragma unroll 1
            for (int x = 0; x < D && mine > 0; x += 32) {
                float o[32];
                tmem_ld32(oa + x, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) buf[(x + y) * kRowTile + row] = o[y];
            }
            buf[D * kRowTile + row] = st.m;
            buf[(D + 1) * kRowTile + row] = st.l;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (stream == 1 || !ok || !active) return;
        const bool both = w.tiles > 1;
        const float m1 = both ? buf[D * kRowTile + row] : -INFINITY, l1 = both ? buf[(D + 1) * kRowTile + row] : 0.f;
        const float m = fmaxf(st.m, m1);
        float f = st.m == -INFINITY ? 0.f : ex2_approx(st.m - m), fo = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
        State sum{m, st.l * f + l1 * fo};
        if (p.n_splits == 1) {
            const float inv = sum.l > 0.f || sum.l != sum.l ? 1.f / sum.l : 0.f;
            f *= inv;
            fo *= inv;
        }
        write_row<D, BITS, ROT>(p, w, oa, w.tiles > 0, valid, r, sum, f, both ? buf + row : nullptr, fo);
        return;
    }
    if (!ok || !active) return;
    const float f = p.n_splits > 1 ? 1.f : (st.l > 0.f || st.l != st.l ? 1.f / st.l : 0.f);
    write_row<D, BITS, ROT>(p, w, oa, w.tiles > 0, valid, r, st, f, nullptr, 0.f);
}

// ------------------------------------------------------------------- kernel --
// ROT: with the transforms of rotated caches (apart, as they take registers and code).
template <int D, int BITS, bool ROT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<D, BITS>;
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    static_assert(offsetof(Bars, slot_empty) == kSlotEmpty && offsetof(Bars, q_full) == kQFull && offsetof(Bars, abort) == kAbort, "addresses");
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);  // (an offset, so that it stays a shared-memory pointer)
    uint8_t* qs = base;
    uint8_t* slots = base + C::kQ;
    uint8_t* ring = slots + C::kSlots * C::kSlot;
    const bool pair = C::kStreams == 2 && p.pair;
    Work w;
    if (!find_work<C::kTile>(p, p.rows_per_item, w)) return;  // the whole CTA
    const int warp = threadIdx.x >> 5;
    if (warp == 16) {
        tmem_alloc(&bars.tmem, 512);
    } else if (threadIdx.x == 17 * 32) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&bars.ring_full[i], 1);
            mbar_init(&bars.ring_empty[i], C::kUnpackWarps);
            mbar_init(&bars.slot_full[i], C::kUnpackWarps);
            mbar_init(&bars.slot_empty[i], pair ? 2 : 1);  // the products that use it
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.o_full[i], 1);
            mbar_init(&bars.drain[i], 1);
        }
        mbar_init(&bars.q_full, C::kStreams * 4);
        mbar_init(&bars.half, 4);
        bars.abort = 0;
        fence_mbarrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // registers: 640 x 96 at launch; 256 x 144 + 256 x 72 + 128 x 48 (one
    // accumulator: 128 x 200 + 128 x 48 + 256 x 72 + 128 x 48)
    if (warp < C::kStreams * 4) {
        regs_raise<C::kStreams == 2 ? 144 : 200>();
        softmax_role<D, BITS, ROT>(p, w, qs, slots, fixed(smem_u32(&bars)), warp >> 2, pair);
    } else if (warp < 8) {
        regs_lower<48>();
    } else if (warp < 16) {
        regs_lower<72>();
        unpack_role<D, BITS>(p, w, fixed(smem_u32(ring)), fixed(smem_u32(slots)), fixed(smem_u32(&bars)), pair);
    } else {
        regs_lower<48>();
        if (warp == 16 || (C::kStreams == 2 && warp == 18)) {
            const uint32_t stream = warp == 18 ? 1 : 0;
            if (w.tiles > 0 && !mma_loop<D, BITS>(p, w, smem_u32(qs), smem_u32(slots), fixed(smem_u32(&bars)), pair, stream)) {
                __syncwarp();
                if (elect_one()) tc_commit(smem_u32(&bars.drain[stream]));  // given up: products in flight end before the CTA leaves
                mbar_wait_bounded(&bars.drain[stream], 0);
            }
        } else if (threadIdx.x == 17 * 32) {
            load_role<D, BITS>(p, w, ring, &bars, pair);
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
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long wid = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int per = p.n * p.group_q;  // rows of a (sequence, kv head)
    const int bh = static_cast<int>(wid / per), flat = static_cast<int>(wid - static_cast<long long>(bh) * per);
    if (bh >= p.batch * p.num_kv_heads) return;
    const int b = bh / p.num_kv_heads, h = bh - b * p.num_kv_heads, i = flat / p.group_q, g = flat - i * p.group_q;
    const int ql = p.q_lens != nullptr ? min(max(p.q_lens[b], 0), p.n) : p.n;
    if (i >= ql) return;
    const int m = flat / p.rows_per_item, r = flat - m * p.rows_per_item;
    const long long part0 = (static_cast<long long>(bh) * p.m_items + m) * p.n_splits;
    float top = -INFINITY;
    for (int s = lane; s < p.n_splits; s += 32) top = fmaxf(top, p.part_m[(part0 + s) * p.rows_per_item + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[E] = {}, l = 0.f;
    for (int s0 = 0; s0 < p.n_splits; s0 += 32) {
        float f = 0.f, pl = 0.f;
        if (s0 + lane < p.n_splits) {
            const long long at = (part0 + s0 + lane) * p.rows_per_item + r;
            const float pm = p.part_m[at];
            f = pm == -INFINITY ? 0.f : ex2_approx(pm - top);
            pl = f == 0.f ? 0.f : f * p.part_l[at];
        }
        const int n = min(32, p.n_splits - s0);
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float fs = __shfl_sync(0xffffffffu, f, s);
            l += __shfl_sync(0xffffffffu, pl, s);
            if (fs == 0.f) continue;  // (an empty part's sums were not written)
            const float* a = p.part_acc + ((part0 + s0 + s) * p.rows_per_item + r) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(fs, a[e], acc[e]);
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
    const long long ctas = static_cast<long long>(p.batch) * p.num_kv_heads * p.m_items * p.n_splits;
    chunk_kernel<D, BITS, ROT><<<static_cast<unsigned>(ctas), kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const ChunkParams& p, cudaStream_t stream) {
    const bool rot = p.rotate_q || (p.rotate_out && p.n_splits == 1);
    cudaError_t e = p.bits == 8 ? (rot ? launch_main<D, 8, true>(p, stream) : launch_main<D, 8, false>(p, stream))
                                : (rot ? launch_main<D, 4, true>(p, stream) : launch_main<D, 4, false>(p, stream));
    if (e != cudaSuccess || p.n_splits == 1) return e;
    const long long rows = static_cast<long long>(p.batch) * p.n * p.num_q_heads, each = kMergeThreads / 32;
    chunk_merge_kernel<D><<<static_cast<unsigned>((rows + each - 1) / each), kMergeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

int chunk_tile_tokens(int head_dim) { return head_dim == 256 ? 64 : 128; }

cudaError_t launch_chunk(const ChunkParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch_dim<64>(p, stream);
    return head_dim == 128 ? launch_dim<128>(p, stream) : launch_dim<256>(p, stream);
}

}  // namespace tq
