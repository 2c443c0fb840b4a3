// What the split kernel of prompt_attn_paged_b8 and verify_attn_shared_b8 (prompt_tc.cuh) and their joining kernels
// (paged_prompt.cu) share: the arguments, the units of work and their deal over the CTAs.
//
// An entity is what has pages and (row, query head) pairs of its own: a sequence (prompts); the pages that a group
// shares with the pairs of all its slots, or a slot with the pages behind those (shared).  For each KV head its pairs are
// taken 256 at a time: a unit, whose work are the tiles (two pages, 128 keys) that its pairs see.  All tiles of
// the call in (entity, head, unit) order are dealt to one CTA an SM by cost.  A run of tiles of one unit in a CTA is a
// segment.  A segment that is its whole unit needs no partial sums (prompts) or leaves them by pair (shared); the
// others leave them in the CTA's two places: 2 c for a segment that continues a unit of the CTA before, 2 c + 1 for one
// that begins a unit which later CTAs continue.
#pragma once

#include <type_traits>

#include "paged_plan.cuh"

#include "kv_prompts.h"

namespace va {
namespace paged {
namespace pr {

constexpr int kPairs = 256;                   // (row, query head) pairs of a unit
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kThreads = 640;
constexpr int kSplits = 8;                    // CTAs that compare a group's table rows, at most
// Costs: of a tile for up to 128 pairs and for more, and of a segment besides its tiles.  From stamps of all CTAs of six calls,
// fitted, in cycles: a tile 3,200 and 4,000, a segment 8,000 to 10,000 in shared calls and 13,000 to 16,500 in prompts (rows go
// straight to the output there).  Measured in us at 8, 9, 10, 12 a segment of shared calls: 8 x 8 slots of 4K 40.2, 39.9,
// 40.3, 41.3, 32 slots behind 16K 51.1, 50.0, 51.6, 51.3; at 15, 18, 21, 24 of prompts: 16K 385, 365, 364, 365, turns 245, 237, 235,
// 236, window 519, 507, 510, 511, 4 x 1K 26.5, 28.3, 25.4, 26.6.
constexpr int kCostOne = 4, kCostTwo = 5;
template <bool kShared>
constexpr int kCostSeg = kShared ? 9 : 21;

// Division by a number that is known before the launch: exact for n d < 2^32.
struct Divisor {
    unsigned d, by;
    __host__ explicit Divisor(unsigned n = 1) : d(n), by(n > 1 ? (unsigned)((0x100000000ull + n - 1) / n) : 0u) {}
    __device__ __forceinline__ unsigned quotient(unsigned n) const { return by ? __umulhi(n, by) : n; }
    __device__ __forceinline__ unsigned rest(unsigned n) const { return n - quotient(n) * d; }
};

struct Args {
    const uint16_t* q;
    const int32_t *first_row, *n_live, *lens, *table;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale, *sink;
    float* part_o;                            // [2 kMaxCtas][256][128]: the CTAs' places
    float2* part_ml;                          // [2 kMaxCtas][256]: (reference, sum)
    int4* begun;                              // prompts: [kMaxCtas]: live rows (-1: none), first row, head, unit of place 2 c + 1
    int* goes_on;                             // [kMaxCtas]: place 2 c is empty (0), a unit's last part (1), a middle one (2)
    float* pair_o;                            // shared: [2][pairs][128], of the shared pages and of the slot's own
    float2* pair_ml;                          // shared: [2][pairs]
    int* first_cta;                           // shared: per unit the CTA that begins it, -1 if that does all of it
    int2* common;                             // shared: [n_groups][kSplits]: first page, pages up to which all agree
    uint16_t* out;
    float* out_lse;
    int32_t* dev_status;
    float scale_log2;                         // |scale| x log2 e
    uint32_t flip;                            // sign bits of q to turn: scale < 0
    int n_seqs, n_rows, n_kv, group, max_pages, n_pages, window, n_ctas;      // n_rows: packed rows, or rows a slot
    int share, n_splits;                      // shared: slots a group, CTAs that compared its rows
    Divisor by_group, by_slots, by_rows;      // group, share + 1, n_rows (shared)
    int shift;                                // costs count in 2^shift, so that their sum fits 30 bits
};

// Pages that a unit's pairs see: [first, first + n), n / 2 tiles rounded up.
struct Unit {
    int first, n, pairs;
    __device__ __forceinline__ int tiles() const { return (n + 1) >> 1; }
    __device__ __forceinline__ int cost_of_tile() const { return pairs > kPairs / 2 ? kCostTwo : kCostOne; }
};

// Length and live rows of a sequence of packed rows.
struct Packed {
    int len, live, first, status;
};
__device__ __forceinline__ Packed load_packed(const Args& a, int b) {
    const Seq s = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
    Packed p;
    p.len = s.len;
    p.live = s.live;
    p.status = s.status;
    p.first = __ldcg(a.first_row + b);
    if (p.live > 0 && (p.first < 0 || p.first > a.n_rows - p.live)) p.status |= VA_DEV_BAD_COUNT;
    if (p.status) p.len = p.live = 0;
    return p;
}

// The pages that a group's slots share: [first, second), from the comparisons.
__device__ __forceinline__ int2 common_of(const Args& a, int g) {
    int2 c = __ldcg(a.common + g * kSplits);
    int y[kSplits];
#pragma unroll
    for (int z = 1; z < kSplits; ++z) y[z] = z < a.n_splits ? __ldcg(&a.common[g * kSplits + z].y) : c.y;
#pragma unroll
    for (int z = 1; z < kSplits; ++z) c.y = min(c.y, y[z]);
    return c;
}

// The units of packed prompts: unit k of a sequence holds pairs 256 k .. (pair = row x group + query head of the group).
__device__ __forceinline__ Unit prompt_unit(int len, int live, const Divisor& group, int window, int k) {
    Unit u;
    const int total = live * (int)group.d, p0 = k * kPairs;
    u.pairs = min(kPairs, total - p0);
    const int start = len - live, hi = start + (int)group.quotient(p0 + u.pairs - 1);
    u.first = window > 0 ? max(0, start + (int)group.quotient(p0) - window + 1) / kPage : 0;
    u.n = hi / kPage + 1 - u.first;
    return u;
}
// The units of what a group shares: pair = (slot in the group x n_rows + row) x group + query head of the group.
__device__ __forceinline__ Unit shared_unit(int2 common, int pairs, int k) {
    Unit u;
    u.pairs = min(kPairs, pairs - k * kPairs);
    u.first = common.x;
    u.n = max(0, common.y - common.x);
    return u;
}
// The unit of a slot's own pages: pair = row x group + query head of the group.
__device__ __forceinline__ Unit slot_unit(int len, int live, int group, int window, int2 common) {
    Unit u;
    u.pairs = live * group;
    u.first = window > 0 ? max(0, len - live - window + 1) / kPage : 0;
    if (common.y > common.x) u.first = max(u.first, common.y);
    u.n = live > 0 ? max(0, (len + kPage - 1) / kPage - u.first) : 0;
    return u;
}

// Number of a shared call's unit, for first_cta.
__device__ __forceinline__ int unit_number(const Args& a, int blocks, int e, int h, int k) {
    const int g = a.by_slots.quotient(e), j = e - g * (a.share + 1), groups = a.n_seqs / a.share;
    return j == 0 ? (g * a.n_kv + h) * blocks + k : groups * a.n_kv * blocks + (g * a.share + j - 1) * a.n_kv + h;
}

struct Place {
    int e, h, k, t;              // entity, head, unit, tile
};

// What an entity's units depend on: a sequence's or slot's length and live rows; a prompt's first row, or the pages that
// the slot's group shares.  (Of an entity that is a group's shared pages only those.)
template <bool kShared>
struct Entity {
    int len, live;
    std::conditional_t<kShared, int2, int> extra;

    __device__ __forceinline__ int blocks(const Args& a, int e) const {
        if constexpr (kShared) return a.by_slots.rest(e) == 0 ? (a.share * a.n_rows * a.group + kPairs - 1) / kPairs : 1;
        else return (int)(((unsigned)live * (unsigned)a.group + kPairs - 1) / kPairs);       // (live below 2^24 + 1, group to 8)
    }
    __device__ __forceinline__ Unit unit(const Args& a, int e, int k) const {
        if constexpr (kShared) {
            if (a.by_slots.rest(e) == 0) return shared_unit(extra, a.share * a.n_rows * a.group, k);
            return slot_unit(len, live, a.group, a.window, extra);
        } else {
            return prompt_unit(len, live, a.by_group, a.window, k);
        }
    }
    __device__ __forceinline__ unsigned cost(const Args& a, int e, int k) const {
        const Unit u = unit(a, e, k);
        return u.n > 0 ? max(1u, ((unsigned)kCostSeg<kShared> + (unsigned)u.tiles() * (unsigned)u.cost_of_tile()) >> a.shift) : 0u;
    }
};

// CTA c's first cost of `total` (below 2^30).
__device__ __forceinline__ unsigned first_cost(unsigned c, unsigned n, unsigned total) {
    return c * (total / n) + c * (total % n) / n;
}

template <bool kShared>
struct Deal {
    static constexpr int kMaxEntities = (kShared ? 2 : 1) * VA_PAGED_MAX_SEQS;
    unsigned pre[kMaxEntities + 1];               // cost of a head before each entity
    unsigned sums[kThreads / 32];
    unsigned long long rows;                      // prompts: all sequences' live rows; 0 before make()
    int len[VA_PAGED_MAX_SEQS];
    std::conditional_t<kShared, signed char, int> live[VA_PAGED_MAX_SEQS];
    std::conditional_t<kShared, int2, int> extra[VA_PAGED_MAX_SEQS];     // a group's common pages; a prompt's first row

    static __device__ __forceinline__ int entities(const Args& a) { return kShared ? a.n_seqs + a.n_seqs / a.share : a.n_seqs; }
    __device__ __forceinline__ Entity<kShared> entity(const Args& a, int e) const {
        Entity<kShared> x;
        if constexpr (kShared) {
            const int g = a.by_slots.quotient(e), j = e - g * (a.share + 1), b = g * a.share + max(j - 1, 0);
            x.len = len[b];
            x.live = live[b];
            x.extra = extra[g];
        } else {
            x.len = len[e];
            x.live = live[e];
            x.extra = extra[e];
        }
        return x;
    }
    // The table row that an entity's pages stand in.
    __device__ __forceinline__ int table_row(const Args& a, int e) const {
        if (!kShared) return e;
        const int g = a.by_slots.quotient(e), j = e - g * (a.share + 1);
        if (j > 0) return g * a.share + j - 1;
        int b = g * a.share;
#pragma unroll 1
        while (live[b] == 0) ++b;                 // (a group that shares pages has live slots)
        return b;
    }

    // The place of `left`, a cost of a head of entity e; all lanes of a warp.
    __device__ __forceinline__ Place place(const Args& a, const Entity<kShared>& x, int e, int h, unsigned left) const {
        Place p = {e, h, 0, 0};
        const int lane = threadIdx.x & 31, n = x.blocks(a, e);
#pragma unroll 1
        for (int k0 = 0;; k0 += 32) {
            const unsigned mine = k0 + lane < n ? x.cost(a, e, k0 + lane) : 0u;
            unsigned upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned t = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += t;
            }
            const unsigned in = __ballot_sync(0xffffffffu, upto > left);
            if (in != 0 || k0 + 32 >= n) {
                const int at = in != 0 ? __ffs(in) - 1 : 31;
                const unsigned inside = left - __shfl_sync(0xffffffffu, upto - mine, at);
                p.k = min(k0 + at, n - 1);
                const unsigned tiles = (unsigned)max(0, (int)(inside << a.shift) - kCostSeg<kShared>);
                p.t = (int)(x.unit(a, e, p.k).cost_of_tile() == kCostTwo ? tiles / kCostTwo : tiles / kCostOne);
                return p;
            }
            left -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    // The place of cost y of all; all lanes of a warp.
    __device__ __forceinline__ Place find(const Args& a, int n, unsigned y) const {
        if (y >= pre[n] * (unsigned)a.n_kv) return {n, 0, 0, 0};
        int lo = 0, hi = n;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] * (unsigned)a.n_kv <= y) lo = mid;
            else hi = mid;
        }
        const unsigned per_head = pre[lo + 1] - pre[lo], rest = y - pre[lo] * (unsigned)a.n_kv;
        return place(a, entity(a, lo), lo, (int)(rest / per_head), rest % per_head);
    }

    // Where this CTA's tiles begin (in `from` of warp 0) and the next one's (in `to`, of warp 1).  Every thread of a CTA calls
    // it, after the launch dependency has resolved.
    __device__ __forceinline__ void make(const Args& a, Place& from, Place& to) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        int status = 0;
#pragma unroll 1
        for (int b = tid; b < a.n_seqs; b += kThreads) {
            if constexpr (kShared) {
                const Seq s = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
                status |= s.status;
                len[b] = s.len;
                live[b] = (signed char)s.live;
            } else {
                const Packed s = load_packed(a, b);
                status |= s.status;
                len[b] = s.len;
                live[b] = s.live;
                extra[b] = s.first;
                atomicAdd(&rows, (unsigned long long)s.live);
            }
        }
        if constexpr (kShared) {
#pragma unroll 1
            for (int g = kThreads - 1 - tid; g < a.n_seqs / a.share; g += kThreads) extra[g] = common_of(a, g);      // (other warps)
        }
        if (status && a.dev_status && blockIdx.x == 0) atomicOr(a.dev_status, status);
        __syncthreads();
        if (!kShared && rows > (unsigned long long)a.n_rows) {
            // (rows of several sequences: the costs could pass 32 bits)
            if (a.dev_status && blockIdx.x == 0 && tid == 0) atomicOr(a.dev_status, VA_DEV_BAD_COUNT);
            for (int b = tid; b < a.n_seqs; b += kThreads) live[b] = 0;
            __syncthreads();
        }
        const int n = entities(a);
        // each entity's cost, for one head: a warp an entity where there are few, or where it has many units
#pragma unroll 1
        for (int e = n > 4 * kThreads / 32 ? tid : n; e < n; e += kThreads) {
            const Entity<kShared> x = entity(a, e);
            pre[e + 1] = x.blocks(a, e) == 1 ? x.cost(a, e, 0) : 0xFFFFFFFFu;
        }
        if (n > 4 * kThreads / 32) __syncthreads();
#pragma unroll 1
        for (int e = warp; e < n; e += kThreads / 32) {
            if (n > 4 * kThreads / 32 && pre[e + 1] != 0xFFFFFFFFu) continue;
            const Entity<kShared> x = entity(a, e);
            const int m = x.blocks(a, e);
            unsigned sum = 0;
#pragma unroll 1
            for (int k = lane; k < m; k += 32) sum += x.cost(a, e, k);
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == 0) pre[e + 1] = sum;
        }
        __syncthreads();
        // their prefix sums
        if (n <= 32) {
            if (warp == 0) {
                unsigned upto = lane < n ? pre[lane + 1] : 0u;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned t = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += t;
                }
                if (lane < n) pre[lane + 1] = upto;
                if (lane == 0) pre[0] = 0;
            }
        } else {
            constexpr int kPer = (kMaxEntities + kThreads - 1) / kThreads;
            const int per = (n + kThreads - 1) / kThreads;
            unsigned mine[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = tid * per + i;
                mine[i] = i < per && e < n ? pre[e + 1] : 0;
                sum += mine[i];
            }
            unsigned upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned t = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += t;
            }
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            unsigned before = upto - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0u);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = tid * per + i;
                if (i < per && e < n) {
                    before += mine[i];
                    pre[e + 1] = before;
                }
            }
            if (tid == 0) pre[0] = 0;
        }
        __syncthreads();
        if (warp < 2) {
            const Place p = find(a, n, first_cost(blockIdx.x + warp, a.n_ctas, pre[n] * (unsigned)a.n_kv));
            if (lane == 0) *(warp == 0 ? &from : &to) = p;
        }
    }
};

// A CTA's segments, in order.  A warp keeps the place of its next one in shared memory, not in registers over its tiles.
struct Segment {
    int e, h, k, t0, t1;         // tiles t0 .. t1 - 1 of the unit
    Unit u;
    bool first, last;            // the segment begins its unit, ends it
    // All lanes of a warp, or one alone that keeps a place of its own.
    template <bool kShared>
    __device__ __forceinline__ bool next(const Deal<kShared>& d, const Args& a, Place& place, const Place& to, bool warp) {
        const int n = Deal<kShared>::entities(a);
        Place p = place;
        if (warp) __syncwarp();
        if (p.e >= n) return false;
        e = p.e;
        h = p.h;
        k = p.k;
        t0 = p.t;
        const bool end = e == to.e && h == to.h && k == to.k;
        const Entity<kShared> x = d.entity(a, e);
        u = x.unit(a, e, k);
        t1 = end ? to.t : u.tiles();
        if (end && t1 <= t0) return false;
        first = t0 == 0;
        last = t1 == u.tiles();
        p.t = 0;
        if (end) {
            p.e = n;
        } else if (++p.k == x.blocks(a, e)) {
            p.k = 0;
            if (++p.h == a.n_kv) {
                p.h = 0;
#pragma unroll 1
                do ++p.e;
                while (p.e < n && d.pre[p.e + 1] == d.pre[p.e]);
            }
        }
        if (!warp || (threadIdx.x & 31) == 0) place = p;
        if (warp) __syncwarp();
        return true;
    }
};

}  // namespace pr
}  // namespace paged
}  // namespace va
