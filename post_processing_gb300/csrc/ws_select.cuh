// ws_select.cuh -- exact selection by unique 64-bit keys: the keys' order and
// the ranking in sorted lists, which the Top-K and the log-probability kernels
// share, and the block's radix select, the 32-key merge and the ranking by
// counting, which the Top-K uses.
//
// A key holds a value's order bits in its upper word (NaN -> -inf, -0 -> +0)
// and the bitwise complement of its index in the lower word, so a larger key
// is a larger value or, for equal values, a lower index.  Keys are unique
// and every real key is larger than 0, which pads the lists.
#pragma once

#include <cstdint>

namespace ws {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kOrderNegInf = 0x007fffffu;   // order_bits(-inf)

__device__ __forceinline__ uint32_t order_bits(float f) {
    uint32_t b = __float_as_uint(f);
    if ((b & 0x7fffffffu) > 0x7f800000u) b = 0xff800000u;   // NaN -> -inf
    if (b == 0x80000000u) b = 0u;                            // -0 -> +0 (ordering only)
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The value of order bits: the float that order_bits maps to them (+0 for
// both zeros, -inf for NaN).
__device__ __forceinline__ float order_value(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ unsigned long long make_key(uint32_t u, uint32_t idx) {
    return ((unsigned long long)u << 32) | (uint32_t)(~idx);
}

__device__ __forceinline__ uint32_t key_index(unsigned long long key) {
    return ~(uint32_t)(key & 0xffffffffull);
}

// Top 32 of two 32-key lists, each sorted descending across the warp (lane
// 0 largest): the lane-wise maximum of one list and the other reversed is a
// bitonic sequence holding the 32 largest keys, and five half-cleaner
// stages sort it descending.
__device__ __forceinline__ unsigned long long merge_top32(unsigned long long a, unsigned long long b) {
    const int lane = threadIdx.x & 31;
    const unsigned long long br = __shfl_sync(kFull, b, 31 - lane);
    unsigned long long c = a > br ? a : br;
#pragma unroll
    for (int j = 16; j >= 1; j >>= 1) {
        const unsigned long long o = __shfl_xor_sync(kFull, c, j);
        c = (lane & j) == 0 ? (c > o ? c : o) : (c < o ? c : o);
    }
    return c;
}

// Exact kth-largest (1-based) of n unique 64-bit keys by radix select, by a
// block of kThreads threads; hist (256) and sel (2) are shared memory.
template <int kThreads, class KeyAt>
__device__ unsigned long long block_kth_largest(KeyAt key_at, int n, int kth, uint32_t* hist, uint32_t* sel) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long prefix = 0, mask = 0;
    uint32_t remaining = (uint32_t)kth;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int base = warp * 32; base < n; base += kThreads) {
            const int i = base + lane;
            uint32_t bin = 256;
            if (i < n) {
                const unsigned long long key = key_at(i);
                if ((key & mask) == prefix) bin = (uint32_t)(key >> shift) & 255u;
            }
            const unsigned peers = __match_any_sync(kFull, bin);
            if (bin < 256 && lane == __ffs(peers) - 1) atomicAdd(&hist[bin], (uint32_t)__popc(peers));
        }
        __syncthreads();
        if (warp == 0) {
            // lane l owns bins 255-8l down to 248-8l
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = hist[255 - 8 * lane - j];
                sum += c[j];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            const uint32_t excl = incl - sum;
            if (excl < remaining && remaining <= incl) {
                uint32_t acc = excl;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (acc < remaining && remaining <= acc + c[j]) {
                        sel[0] = 255u - 8u * lane - j;
                        sel[1] = remaining - acc;
                    }
                    acc += c[j];
                }
            }
        }
        __syncthreads();
        prefix |= (unsigned long long)sel[0] << shift;
        mask |= 0xffull << shift;
        remaining = sel[1];
        __syncthreads();
    }
    return prefix;
}

// Ranks the `cnt` unique candidates in keys[] (shared memory) and calls
// emit(rank, key) for ranks below `kk`; a candidate's rank is the number of
// larger keys.  One thread per candidate: splitting a candidate's count over
// several threads measured slower on GB300 (64 x 1000: 4.0 against 3.3 us).
template <int kThreads, class Emit>
__device__ __forceinline__ void rank_and_emit(const unsigned long long* keys, uint32_t cnt, int kk, Emit emit) {
    for (uint32_t i = threadIdx.x; i < cnt; i += kThreads) {
        const unsigned long long key = keys[i];
        int rank = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < cnt; ++j) rank += (keys[j] > key) ? 1 : 0;
        if (rank < kk) emit(rank, key);
    }
}

// The number of keys larger than `key` in kLists sorted lists of 32 (shared
// memory): a branch-free binary search in each, all in lockstep so that
// their loads overlap.
template <int kLists>
__device__ __forceinline__ int rank_in_lists(const unsigned long long (*lists)[32], unsigned long long key) {
    int lo[kLists];
#pragma unroll
    for (int c = 0; c < kLists; ++c) lo[c] = 0;
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1)
#pragma unroll
        for (int c = 0; c < kLists; ++c) lo[c] += lists[c][lo[c] + step - 1] > key ? step : 0;
    int rank = 0;
#pragma unroll
    for (int c = 0; c < kLists; ++c) rank += lo[c] + (lists[c][lo[c]] > key ? 1 : 0);
    return rank;
}

}  // namespace ws
