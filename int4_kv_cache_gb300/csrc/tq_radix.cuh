// tq_radix.cuh -- the n-th largest of a CTA's keys, shared by the block selection
// and the eviction.
#pragma once

#include <stdint.h>

namespace tq {

namespace {

constexpr int kFew = 32;  // keys that a warp ranks by itself

// The n-th largest (n >= 1) of the keys visit() hands out, all of them in [lo,
// hi] and `count` in number, by digits of eight bits from the highest in which
// lo and hi differ, until kFew keys or fewer share the digits so far; those are
// gathered and ranked directly.  `above`: how many keys are larger.  Every
// thread of the CTA calls with hist zeroed (both halves) a barrier ago; visit(f)
// calls f(key) for this thread's keys.
template <int THREADS, typename K, typename Visit>
__device__ __forceinline__ K nth_largest(int n, int count, K lo, K hi, Visit visit, uint32_t (*hist)[256], int& above) {
    __shared__ K few[kFew];
    __shared__ int n_few;
    const int lane = threadIdx.x & 31;
    above = 0;
    const K diff = lo ^ hi;
    int bits;  // the low bits in which keys may differ
    if constexpr (sizeof(K) == 8) bits = diff == 0 ? 0 : 64 - __clzll(static_cast<long long>(diff));
    else bits = 32 - __clz(static_cast<int>(diff));
    const K ones = ~static_cast<K>(0);
    K mask = bits == static_cast<int>(sizeof(K) * 8) ? 0 : ones << bits;
    K value = hi & mask;
    if (threadIdx.x == 0) n_few = 0;
    __syncthreads();
    auto rank_few = [&]() -> K {  // of the keys that share the digits so far
        visit([&](K k) {
            if ((k & mask) == value) {
                const int at = atomicAdd(&n_few, 1);
                if (at < kFew) few[at] = k;
            }
        });
        __syncthreads();
        const int m = min(n_few, kFew);
        const K mine = lane < m ? few[lane] : 0;
        int greater = 0, equal = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) {
            const K o = few[j];
            greater += o > mine ? 1 : 0;
            equal += o == mine ? 1 : 0;
        }
        const int need = n - above;
        const uint32_t it = __ballot_sync(0xffffffffu, lane < m && greater < need && need <= greater + equal);
        const int at = it != 0 ? __ffs(it) - 1 : 0;
        above += __shfl_sync(0xffffffffu, greater, at);
        return __shfl_sync(0xffffffffu, mine, at);
    };
    if (bits > 0 && count <= kFew) return rank_few();
    for (int pass = 0; bits > 0; ++pass) {
        const int take = bits < 8 ? bits : 8, shift = bits - take, h = pass & 1;
        visit([&](K k) {
            if ((k & mask) == value) atomicAdd(&hist[h][static_cast<uint32_t>(k >> shift) & ((1u << take) - 1u)], 1u);
        });
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += THREADS) hist[h ^ 1][i] = 0;  // read a barrier ago
        // Every warp finds the digit: lane l holds bins 255 - 8 l .. 248 - 8 l,
        // counts from the largest down.  (Their sum in an order of the lane's
        // own, so that the lanes' banks differ.)
        const uint32_t* bins = &hist[h][255 - 8 * lane];
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += bins[-((j + (lane >> 2)) & 7)];
        uint32_t before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += o;
        }
        before -= sum;
        const uint32_t want = static_cast<uint32_t>(n - above);
        uint32_t bin = 0, ahead = 0, here = 0;
        const bool mine = before < want && want <= before + sum;
        if (mine) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t c = bins[-j];
                if (before < want && want <= before + c) {
                    bin = 255 - 8 * lane - j;
                    ahead = before;
                    here = c;
                }
                before += c;
            }
        }
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        const int src = who != 0 ? __ffs(who) - 1 : 0;
        bin = __shfl_sync(0xffffffffu, bin, src);
        above += static_cast<int>(__shfl_sync(0xffffffffu, ahead, src));
        here = __shfl_sync(0xffffffffu, here, src);
        value |= static_cast<K>(bin) << shift;
        bits = shift;
        mask = shift == 0 ? ones : ones << shift;
        if (bits > 0 && here <= kFew) return rank_few();  // the same for the CTA
        __syncthreads();  // the other half is zero, this one has been read
    }
    return value;
}

}  // namespace

}  // namespace tq
