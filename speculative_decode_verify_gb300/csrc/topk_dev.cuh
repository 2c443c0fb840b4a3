// Ranking of logits, shared by the sampler and beam search: 64-bit keys in candidate order, and the k best keys of
// an 8,192-logit tile.
#pragma once

#include <cstdint>

#include "spec_sample.h"

namespace va {
namespace smp {

constexpr int kTileLogits = VA_SAMPLE_TILE;   // 8192
constexpr int kThreads = 256;
constexpr int kPerThread = kTileLogits / kThreads;   // 32
constexpr int kMaxK = VA_SAMPLE_MAX_K;        // 32
constexpr int kMaxCand = 256;                 // candidates ranked by counting; more take the slow path

// Order-preserving image of a float (NaN lowest, -0 == +0).
__device__ __forceinline__ uint32_t ord_bits(float f) {
    if (f != f) return 0u;
    uint32_t b = __float_as_uint(f);
    if ((b & 0x7FFFFFFFu) == 0u) b = 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ord_to_float(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint64_t make_key(float f, int idx) {
    return ((uint64_t)ord_bits(f) << 32) | (uint32_t)(~(uint32_t)idx);
}
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(~(uint32_t)(key & 0xFFFFFFFFu)); }

__device__ __forceinline__ uint64_t warp_max_u64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        v = w > v ? w : v;
    }
    return v;
}

// Sort the 32 keys of a warp, largest first (bitonic network over the lanes); returns this lane's key.
__device__ __forceinline__ uint64_t warp_sort_desc_u64(uint64_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, v, stride);
            const bool lower = (lane & stride) == 0;           // this lane holds the lower index of the pair
            const bool desc = (lane & size) == 0;              // this block of the network sorts descending
            const bool keep_big = lower == desc;
            v = keep_big ? (o > v ? o : v) : (o < v ? o : v);
        }
    }
    return v;
}

// k-th largest (1-based) of 256 distinct keys held one per thread.  Each warp sorts its 32 keys; the rank
// of a key is the number of larger keys in every warp's sorted list (a binary search each).
inline __device__ uint64_t block_kth_largest_u64(uint64_t v, int k, uint64_t* lists /*[8][32]*/, uint64_t* out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) *out = 0ull;   // the answer when it is one of several equal zero (empty-thread) keys
    const uint64_t s = warp_sort_desc_u64(v, lane);
    lists[warp * 32 + lane] = s;
    __syncthreads();
    // in every other list, the count of entries > s (lists are descending): a branchless binary search,
    // the eight searches interleaved step by step
    int cnt[kThreads / 32];
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) cnt[w] = 0;
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            if (lists[w * 32 + cnt[w] + step - 1] > s) cnt[w] += step;
    }
    int rank = lane;   // larger keys in this warp's own list
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        // cnt counts entries > s among the first 31; the last entry decides the 32nd
        const int c = cnt[w] + ((cnt[w] == 31 && lists[w * 32 + 31] > s) ? 1 : 0);
        rank += (w == warp) ? 0 : c;
    }
    if (rank == k - 1) *out = s;
    __syncthreads();
    const uint64_t r = *out;
    __syncthreads();
    return r;
}

// Largest key over the block (each thread offers one).
inline __device__ uint64_t block_max_u64(uint64_t v, uint64_t* red /*[8]*/) {
    v = warp_max_u64(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t m = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = red[w] > m ? red[w] : m;
    __syncthreads();
    return m;
}

// The k largest keys of a tile of 256 threads x 32 keys, largest first, to out[0..k-1] (0 past the tile's keys).
// full_warps: how many of the block's warps (the first ones) have a logit in every thread.  Smem holds cand
// (kMaxCand keys), lists, red, wmin, tau and n_cand; every thread of the block calls it.
template <class Smem>
__device__ __forceinline__ void collect_tile(const uint64_t (&key)[kPerThread], int full_warps, int k, Smem& sm,
                                             uint64_t* __restrict__ out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t mx[kPerThread / 2];   // the thread maximum as a tree (short dependency chain)
#pragma unroll
    for (int i = 0; i < kPerThread / 2; ++i) mx[i] = key[2 * i] > key[2 * i + 1] ? key[2 * i] : key[2 * i + 1];
#pragma unroll
    for (int w = kPerThread / 4; w >= 1; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) mx[i] = mx[i] > mx[i + w] ? mx[i] : mx[i + w];
    const uint64_t tmax = mx[0];
    if (tid == 0) sm.n_cand = 0;
    // threshold tau: a lower bound of the tile's k-th largest key, so that every key of the tile's top k is
    // at or above it.  With f warps whose 32 threads all hold logits, take j = ceil(k / f): in each such
    // warp, the j-th largest distinct value among its thread maxima (one warp-wide max per round, the
    // lanes at the maximum dropped), then the minimum over those warps.  Each of the f warps has at least
    // j threads whose maximum is at or above tau, so at least k distinct keys are: the k-th largest is.
    // Only the value bits are compared; all keys with the value are kept.  A tile with fewer than 32
    // threads of logits takes the exact k-th largest thread maximum (an empty thread offers key 0, below
    // every logit; a tile with fewer than k logits gets 0).
    uint64_t tau;
    if (full_warps > 0) {
        const int j = (k + full_warps - 1) / full_warps;
        uint32_t v = (uint32_t)(tmax >> 32), m = 0u;
        for (int r = 0; r < j; ++r) {
            m = __reduce_max_sync(0xffffffffu, v);
            v = (v == m) ? 0u : v;
        }
        if (lane == 0) sm.wmin[warp] = warp < full_warps ? m : 0xFFFFFFFFu;
        __syncthreads();
        uint32_t t = 0xFFFFFFFFu;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t = min(t, sm.wmin[w]);
        tau = (uint64_t)t << 32;
    } else {
        tau = block_kth_largest_u64(tmax, k, sm.lists, &sm.tau);
    }
    // compact the keys at or above the threshold: per-thread count, warp scan, one atomic per warp
    unsigned mine = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) mine |= (key[i] != 0ull && key[i] >= tau) ? (1u << i) : 0u;
    const int cnt = __popc(mine);
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    int wbase = 0;
    if (lane == 31 && incl > 0) wbase = atomicAdd(&sm.n_cand, incl);
    wbase = __shfl_sync(0xffffffffu, wbase, 31);
    int slot = wbase + incl - cnt;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if ((mine >> i) & 1u) {
            if (slot < kMaxCand) sm.cand[slot] = key[i];
            ++slot;
        }
    }
    __syncthreads();
    const int nc = sm.n_cand;
    if (nc <= kMaxCand) {
        // rank by counting: candidate c goes to position (number of larger candidates) if that is < k
        for (int c = tid; c < nc; c += kThreads) {
            const uint64_t kc = sm.cand[c];
            int rank = 0;
#pragma unroll 8
            for (int o = 0; o < nc; ++o) rank += sm.cand[o] > kc;
            if (rank < k) out[rank] = kc;
        }
        for (int r = nc + tid; r < k; r += kThreads) out[r] = 0ull;   // fewer than k logits in the tile
    } else {
        // many equal values at the threshold: k rounds of block-wide maximum over every logit
        uint64_t taken = ~0ull;   // keys below this one remain
        for (int r = 0; r < k; ++r) {
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) m = (key[i] < taken && key[i] > m) ? key[i] : m;
            const uint64_t best = block_max_u64(m, sm.red);
            if (tid == 0) out[r] = best;
            taken = best;
        }
    }
}

}  // namespace smp
}  // namespace va
