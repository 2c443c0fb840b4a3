// prompt_attn_paged_b8 and verify_attn_shared_b8: the calls, the kernel that finds what a group's slots share, and the
// launches that join what the split kernel (prompt_tc.cuh) left in parts.
//
// Joining reads two parts a CTA at most, 128 KB each: 5 us of a small call, 12 of a 16K prompt's 353.  Comparing a group's
// table rows takes 3 to 4 us (16K positions of 32 slots: 8,192 entries, one launch ahead of the split).
#include <algorithm>
#include <cmath>

#include "prompt_plan.cuh"

namespace va {
namespace paged {
namespace pr {

cudaError_t launch_e4m3(const Args& a, bool shared, cudaStream_t stream);
cudaError_t launch_int8(const Args& a, bool shared, cudaStream_t stream);

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kCommonThreads = 1024, kCommonPages = 128;      // threads; pages that a CTA compares at a time
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------------------------------------ shared pages
// CTA (g, z): pages z, z + gridDim.y, .. (128 at a time, eight threads each) of those that every live row of group g sees to their end: the first
// of them in which the table rows of its live slots do not agree.  No pages where fewer than two slots are live.
__global__ void __launch_bounds__(kCommonThreads) common_kernel(const Args a) {
    __shared__ int least[4];        // first live slot, live slots (negative), pages, first page
    __shared__ unsigned is_live[VA_PAGED_MAX_SEQS / 32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, b0 = blockIdx.x * a.share;
    if (tid < 4) least[tid] = tid == 1 ? 0 : 0x7FFFFFFF;
    __syncthreads();
    for (int j0 = tid - lane; j0 < a.share; j0 += kCommonThreads) {
        Seq s = {0, 0, 0};
        if (j0 + lane < a.share) s = load_seq(a.lens, a.n_live, b0 + j0 + lane, a.n_rows, a.max_pages);
        const bool on = s.live > 0;
        const unsigned some = __ballot_sync(0xffffffffu, on);
        const int pages = __reduce_min_sync(0xffffffffu, on ? (s.len - s.live + 1) / kPage : 0x7FFFFFFF);
        const int first = __reduce_min_sync(0xffffffffu, on && a.window > 0 ? max(0, s.len - s.live - a.window + 1) / kPage : on ? 0 : 0x7FFFFFFF);
        if (lane == 0) {
            is_live[j0 / 32] = some;
            if (some) atomicMin(&least[0], j0 + __ffs(some) - 1);
            atomicSub(&least[1], __popc(some));
            atomicMin(&least[2], pages);
            atomicMin(&least[3], first);
        }
    }
    __syncthreads();
    const int lead = least[0], limit = -least[1] < 2 ? 0 : least[2], first = limit > 0 ? least[3] : 0;     // (no live slot: no first)
    __syncthreads();
    if (tid == 0) least[2] = limit;
    __syncthreads();
    for (int x0 = first + blockIdx.y * kCommonPages; x0 < limit; x0 += gridDim.y * kCommonPages) {
        const int x = x0 + (tid & (kCommonPages - 1));
        if (x < limit) {
            const int32_t* row = a.table + (size_t)b0 * a.max_pages + x;
            const int entry = __ldcg(row + (size_t)lead * a.max_pages);
            bool same = true;
#pragma unroll 4
            for (int j = lead + 1 + tid / kCommonPages; j < a.share; j += kCommonThreads / kCommonPages) {
                // (the table rows of slots without live rows may hold anything)
                const int other = __ldcg(row + (size_t)j * a.max_pages);
                same = same && (other == entry || !((is_live[j >> 5] >> (j & 31)) & 1));
            }
            if (!same) atomicMin(&least[2], x);
        }
        __syncthreads();
        if (least[2] < limit) break;
        __syncthreads();
    }
    __syncthreads();
    if (tid == 0) a.common[blockIdx.x * kSplits + blockIdx.y] = make_int2(first, least[2]);
}

// ------------------------------------------------------------------------------------------------ joining
// What a row's parts add up to: four dimensions a lane.
struct Sum {
    float4 o;
    float m, l;
};
__device__ __forceinline__ Sum no_sum() { return {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.0f}; }
// (a part without a weight may still hold a sum that is no number)
__device__ __forceinline__ float part_weight(const float2& ml, float top) {
    return ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.0f) : exp2f(ml.x - top);
}

// Adds the parts of pair `col` in the places list[first], list[first + step], ..: kFlight of them on their way at once.
template <int kFlight>
__device__ __forceinline__ void add_places(const Args& a, Sum& s, const int* list, int n, int first, int step, int col) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int k = first; k < n; k += step * kFlight) {
        float4 v[kFlight];
        float2 ml[kFlight];
        float top = s.m;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            ml[i] = make_float2(-INFINITY, 0.0f);
            if (k + i * step < n) {
                const size_t at = (size_t)list[k + i * step] * kPairs + col;
                ml[i] = __ldcg(a.part_ml + at);
                v[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * kD) + lane);
            }
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) top = fmaxf(top, ml[i].x);
        const float was = s.m == -INFINITY ? 0.0f : exp2f(s.m - top);
        s.m = top;
        s.l = s.l != s.l ? s.l : s.l * was;
        s.o = make_float4(s.o.x * was, s.o.y * was, s.o.z * was, s.o.w * was);
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const float by = part_weight(ml[i], top);
            s.l = fmaf(by, ml[i].y, s.l);
            s.o.x = fmaf(by, v[i].x, s.o.x);
            s.o.y = fmaf(by, v[i].y, s.o.y);
            s.o.z = fmaf(by, v[i].z, s.o.z);
            s.o.w = fmaf(by, v[i].w, s.o.w);
        }
    }
}
__device__ __forceinline__ void add_sum(Sum& s, const float4& o, const float2& ml) {
    const float top = fmaxf(s.m, ml.x), was = s.m == -INFINITY ? 0.0f : exp2f(s.m - top), by = part_weight(ml, top);
    s.l = fmaf(by, ml.y, s.l != s.l ? s.l : s.l * was);
    s.m = top;
    s.o = make_float4(fmaf(by, o.x, s.o.x * was), fmaf(by, o.y, s.o.y * was), fmaf(by, o.z, s.o.z * was), fmaf(by, o.w, s.o.w * was));
}
// The places of the parts of the unit that CTA c of the split kernel begins and later ones continue (a CTA without a share may
// lie between), in order; a warp's lanes together.  `kinds` is goes_on.
__device__ __forceinline__ int list_places(const int* kinds, int n_ctas, int c, int* list) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (lane == 0) list[0] = 2 * c + 1;
    int n = 1;
#pragma unroll 1
    for (int c0 = (c + 1) & ~31; c0 < n_ctas; c0 += 32) {
        const int i = c0 + lane, kind = i > c && i < n_ctas ? kinds[i] : 0;
        const unsigned end = __ballot_sync(0xffffffffu, kind == 1);
        const unsigned upto = end != 0 ? (2u << (__ffs(end) - 1)) - 1u : 0xffffffffu;
        const unsigned parts = __ballot_sync(0xffffffffu, kind != 0) & upto;
        if ((parts >> lane) & 1) list[n + __popc(parts & ((1u << lane) - 1u))] = 2 * i;
        n += __popc(parts);
        if (end != 0) break;
    }
    __syncwarp();
    return n;
}
__device__ __forceinline__ void write_row(const Args& a, const Sum& s, size_t row, int head) {
    const int lane = threadIdx.x & 31;
    const Finish f = finish(s.m, s.l, a.sink, head);
    store_row(a.out + row * kD + 4 * lane, make_float4(s.o.x * f.by, s.o.y * f.by, s.o.z * f.by, s.o.w * f.by));
    if (lane == 0 && a.out_lse) a.out_lse[row] = f.lse;
}
// The eight warps' sums, in warp 0.
struct Meeting {
    float4 o[kJoinWarps][32];
    float2 ml[kJoinWarps];
};
__device__ __forceinline__ void meet(Meeting& mt, Sum& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    mt.o[warp][lane] = s.o;
    if (lane == 0) mt.ml[warp] = make_float2(s.m, s.l);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) add_sum(s, mt.o[w][lane], mt.ml[w]);
}

// Prompts: the pairs of the units that the split kernel left in parts, 256 a unit.  Of few units a pair a CTA, whose warps
// share its (then many) parts; of more four pairs a warp, four parts of each on their way at once, and what belongs to a pair and a
// part alone computed by one lane (16K prompt: 21 us of the call with each lane computing all of it, 12 so).
__global__ void __launch_bounds__(kJoinThreads) join_prompt_kernel(const Args a) {
    __shared__ int kinds[kMaxCtas], cta_of[kMaxCtas], n_units;
    __shared__ int4 units[kMaxCtas];                       // live rows, first row, head, unit
    __shared__ int list[kJoinWarps][kMaxCtas + 1];
    __shared__ Meeting mt;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < a.n_ctas) {
        kinds[tid] = __ldcg(a.goes_on + tid);
        units[tid] = __ldcg(a.begun + tid);
    }
    __syncthreads();
    if (warp == 0) {
        // the CTAs that have begun a unit and not ended it, in order
        int n = 0;
        for (int i = lane; i < (a.n_ctas + 31) / 32 * 32; i += 32) {
            const bool on = i < a.n_ctas && units[i].x >= 0;
            const unsigned some = __ballot_sync(0xffffffffu, on);
            if (on) cta_of[n + __popc(some & ((1u << lane) - 1u))] = i;
            n += __popc(some);
        }
        if (lane == 0) n_units = n;
    }
    __syncthreads();
    const int n_pairs = n_units * kPairs, heads = a.n_kv * a.group;
    if (n_pairs <= 16 * a.n_ctas) {
        for (int item = blockIdx.x; item < n_pairs; item += gridDim.x) {
            const int c = cta_of[item / kPairs], i = item % kPairs, pair = units[c].w * kPairs + i;
            const int r = a.by_group.quotient(pair), head = units[c].z * a.group + pair - r * a.group;
            if (r >= units[c].x) continue;
            Sum sum = no_sum();
            const int n = list_places(kinds, a.n_ctas, c, list[warp]);
            add_places<8>(a, sum, list[warp], n, warp, kJoinWarps, i);
            meet(mt, sum);
            if (warp == 0) write_row(a, sum, (size_t)(units[c].y + r) * heads + head, head);
        }
        return;
    }
    // what belongs to a pair and a part alone is a lane's: pair lane % 4, part lane / 4 % 4
    const int mine4 = lane & 3, part = (lane >> 2) & 3;
    for (int item = blockIdx.x * kJoinWarps + warp; item < n_pairs / 4; item += gridDim.x * kJoinWarps) {
        const int c = cta_of[item / (kPairs / 4)], i0 = item % (kPairs / 4) * 4, pair0 = units[c].w * kPairs + i0;
        if ((int)a.by_group.quotient(pair0) >= units[c].x) continue;
        const int n = list_places(kinds, a.n_ctas, c, list[warp]);
        float m = -INFINITY, l = 0.0f;
        float4 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = 0; k < n; k += 4) {
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (k + part < n) ml = __ldcg(a.part_ml + (size_t)list[warp][k + part] * kPairs + i0 + mine4);
            float4 v[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[i][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k + i < n) v[i][q] = __ldcg(reinterpret_cast<const float4*>(a.part_o + ((size_t)list[warp][k + i] * kPairs + i0 + q) * kD) + lane);
                }
            float top = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, 4));
            top = fmaxf(m, fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8)));
            const float by = part_weight(ml, top), was = m == -INFINITY ? 0.0f : exp2f(m - top);
            float sum = by * ml.y;
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            l = fmaf(l, was, sum);
            m = top;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float less = __shfl_sync(0xffffffffu, was, q);
                o[q] = make_float4(o[q].x * less, o[q].y * less, o[q].z * less, o[q].w * less);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = __shfl_sync(0xffffffffu, by, 4 * i + q);
                    o[q] = make_float4(fmaf(z, v[i][q].x, o[q].x), fmaf(z, v[i][q].y, o[q].y), fmaf(z, v[i][q].z, o[q].z), fmaf(z, v[i][q].w, o[q].w));
                }
            }
        }
        const int r = a.by_group.quotient(pair0 + mine4), head = units[c].z * a.group + pair0 + mine4 - r * a.group;
        const Finish f = finish(m, l, a.sink, head);
        if (lane < 4 && r < units[c].x && a.out_lse) a.out_lse[(size_t)(units[c].y + r) * heads + head] = f.lse;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int rq = __shfl_sync(0xffffffffu, r, q), hq = __shfl_sync(0xffffffffu, head, q);
            const float z = __shfl_sync(0xffffffffu, f.by, q);
            if (rq < units[c].x)
                store_row(a.out + ((size_t)(units[c].y + rq) * heads + hq) * kD + 4 * lane,
                          make_float4(o[q].x * z, o[q].y * z, o[q].z * z, o[q].w * z));
        }
    }
}

// Shared: each row's parts of the shared pages and of its slot's own.  Of few rows one a CTA, of more one a warp.
__global__ void __launch_bounds__(kJoinThreads) join_shared_kernel(const Args a) {
    __shared__ int kinds[kMaxCtas];
    __shared__ int list[kJoinWarps][kMaxCtas + 1];
    __shared__ Meeting mt;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = a.n_rows * a.group;
    const int total = a.n_seqs * a.n_kv * pairs;
    const bool together = total <= (int)gridDim.x;
    const int item = min(together ? (int)blockIdx.x : (int)blockIdx.x * kJoinWarps + warp, total - 1);     // (the last twice over)
    // rows in the order of out: (slot, row, head); all that is known of one is on its way at once
    const int heads = a.n_kv * a.group, head = item % heads, row = item / heads, b = a.by_rows.quotient(row), r = row - b * a.n_rows;
    const int h = a.by_group.quotient(head), pair = r * a.group + head - h * a.group, g = b / a.share, j = b - g * a.share;
    const int blocks = (a.share * pairs + kPairs - 1) / kPairs, shared_pair = j * pairs + pair;
    const int c_shared = __ldcg(a.first_cta + unit_number(a, blocks, g * (a.share + 1), h, shared_pair / kPairs));
    const int c_own = __ldcg(a.first_cta + unit_number(a, blocks, g * (a.share + 1) + j + 1, h, 0));
    const int2 common = common_of(a, g);
    const Seq s = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
    if (tid < a.n_ctas) kinds[tid] = __ldcg(a.goes_on + tid);
    __syncthreads();
    if (r >= s.live) {
        if (together && warp != 0) return;
        reinterpret_cast<uint2*>(a.out + (size_t)item * kD)[lane] = make_uint2(0u, 0u);
        if (lane == 0 && a.out_lse) a.out_lse[item] = -INFINITY;
        return;
    }
    Sum sum = no_sum();
#pragma unroll 1
    for (int own = 0; own < 2; ++own) {
        const int at = own ? pair : shared_pair, c = own ? c_own : c_shared;
        const Unit u = own ? slot_unit(s.len, s.live, a.group, a.window, common) : shared_unit(common, a.share * pairs, at / kPairs);
        if (u.n == 0) continue;
        if (c >= 0 && c < a.n_ctas) {             // (a split that gave up may have left anything)
            const int n = list_places(kinds, a.n_ctas, c, list[warp]);
            add_places<8>(a, sum, list[warp], n, together ? warp : 0, together ? kJoinWarps : 1, at % kPairs);
        } else if (!together || warp == own) {
            const size_t i = (own ? (size_t)total : 0) + item;
            add_sum(sum, __ldcg(reinterpret_cast<const float4*>(a.pair_o + i * kD) + lane), __ldcg(a.pair_ml + i));
        }
    }
    if (together) meet(mt, sum);
    if (!together || warp == 0) write_row(a, sum, item, head);
}

// ------------------------------------------------------------------------------------------------ the calls
// Workspaces: the CTAs' places and records; shared calls behind them the groups' pages, the units' CTAs and the pairs' sums.
struct Layout {
    size_t part_ml, begun, goes_on, common, first_cta, pair_ml, pair_o, bytes;
};
static Layout layout(int n_seqs, int n_rows, int n_kv, int group, bool shared) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout w = {};
    w.part_ml = sizeof(float) * 2 * kMaxCtas * kPairs * kD;
    w.begun = w.part_ml + sizeof(float2) * 2 * kMaxCtas * kPairs;
    w.goes_on = w.begun + sizeof(int4) * kMaxCtas;
    w.common = up(w.goes_on + sizeof(int) * kMaxCtas);
    w.first_cta = w.pair_ml = w.pair_o = w.bytes = w.common;
    if (!shared) return w;
    const size_t pairs = (size_t)n_seqs * n_rows * n_kv * group;
    // units: one a slot and head, and of each group's pairs a 256th, rounded up (at most one a slot more)
    const size_t units = (size_t)n_seqs * n_kv * 2 + pairs / kPairs + 1;
    w.first_cta = w.common + sizeof(int2) * kSplits * (size_t)n_seqs;
    w.pair_ml = up(w.first_cta + sizeof(int) * units);
    w.pair_o = up(w.pair_ml + sizeof(float2) * 2 * pairs);
    w.bytes = w.pair_o + sizeof(float) * 2 * pairs * kD;
    return w;
}

// So that the costs of `units` units of up to max_pages pages add up to less than 2^30.
static int cost_shift(long long units, int max_pages) {
    const long long most = kCostSeg<false> + (long long)kCostTwo * (max_pages / 2 + 1);
    int shift = 0;
    while (units * ((most >> shift) + 1) >= (1ll << 30)) ++shift;
    return shift;
}

// Whether a call of verify_attn_shared_b8 is better off slot by slot, by the sizes alone (lengths are on the device:
// max_pages stands for them, or what a window leaves).  In ns, fitted to both ways' times: verify_attn_paged_b8 takes for a
// page and head of each slot one and one more for each 8 (row, query head) pairs, over all SMs; sharing takes 6 us for its
// launches, 33 for each slot and head, and 6 (to 128 pairs of a group) or 9 (to 256) for each page and head of a group.
// Measured (us, slot by slot and shared): 2 x 4 slots, 1 head, 6 pairs, 4K positions 12.2 and 17.5; 8 slots, 8 heads, 6 pairs,
// 4K 19.3 and 22.3, 8K 26.2 and 26.1, 16K 40.8 and 31.0; 4 slots, 8 heads, 4 pairs, 16K 25.2 and 29.6, 64K 70.6 and 67.2; 4
// slots, 4 heads, 64 pairs, 16K 50.0 and 30.1; 4 x 16 slots, 8 heads, 4 pairs, 1K 36.9 and 45.6, 2K 51.6 and 46.9; 32 x 4
// slots, 8 heads, 4 pairs, 1K 65.8 and 104.6, 4K 174.6 and 173.8.  Where the table is wider than the lengths need the rule errs
// towards sharing: 2 x 4 slots, 1 head, 6 pairs, 1K 11.2 us by a table of 18 columns, 17.2 by one of 2,048 (8 x 8 slots, 4 heads, 4
// pairs, 4K 38.3 and 39.2).  Groups that share nothing (known on the device alone): 8 x 8 slots, 4 heads, 4 pairs, 4K 54.0 and
// 117.8; 32 slots, 8 heads, 6 pairs, 16K 169.6 and 408.4; 8 slots, 8 heads, 6 pairs, 128K 318 and 778; 8 x 8 slots, 1 head, 6 pairs, 32K
// 90.6 and 210.4; 2 x 4 slots, 1 head, 48 pairs, 64K 64.0 and 68.4; 4 x 8 slots, 2 heads, 64 pairs, 8K 90.3 and 70.7.
static bool slot_by_slot(long long n_seqs, int n_rows, int n_kv, int group, int share, int max_pages, int window) {
    const long long pages = window > 0 ? std::min<long long>(max_pages, ((long long)window + n_rows) / kPage + 2) : max_pages;
    const int pairs = n_rows * group, all = pairs * share;
    const long long apart = n_seqs * n_kv * pages * (1 + (pairs + 7) / 8);
    const long long tile = 9 * (all / kPairs) + (all % kPairs > kPairs / 2 ? 9 : all % kPairs > 0 ? 6 : 0);
    return apart <= 6000 + 33 * n_seqs * n_kv + n_seqs / share * n_kv * pages * tile;
}

static void place(Args& a, void* workspace, const Layout& w) {
    char* p = static_cast<char*>(workspace);
    a.part_o = reinterpret_cast<float*>(p);
    a.part_ml = reinterpret_cast<float2*>(p + w.part_ml);
    a.begun = reinterpret_cast<int4*>(p + w.begun);
    a.goes_on = reinterpret_cast<int*>(p + w.goes_on);
    a.common = reinterpret_cast<int2*>(p + w.common);
    a.first_cta = reinterpret_cast<int*>(p + w.first_cta);
    a.pair_ml = reinterpret_cast<float2*>(p + w.pair_ml);
    a.pair_o = reinterpret_cast<float*>(p + w.pair_o);
}

}  // namespace pr
}  // namespace paged
}  // namespace va

extern "C" {

size_t va_prompt_workspace_bytes(int n_seqs, int n_tokens, int n_kv_heads, int group) {
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || n_tokens < 1 || n_tokens > VA_MAX_TOKENS || n_kv_heads < 1 ||
        n_kv_heads > VA_PAGED_MAX_KV_HEADS || group < 1 || group > VA_PAGED_MAX_GROUP)
        return 0;
    return va::paged::pr::layout(n_seqs, n_tokens, n_kv_heads, group, false).bytes;   // two parts a CTA, whatever the batch
}

size_t va_shared_workspace_bytes(int n_seqs, int n_rows, int n_kv_heads, int group) {
    if (va_paged_workspace_bytes(n_seqs, n_rows, n_kv_heads, group) == 0) return 0;
    return std::max(va::paged::pr::layout(n_seqs, n_rows, n_kv_heads, group, true).bytes,
                    va_paged_workspace_bytes(n_seqs, n_rows, n_kv_heads, group));
}

va_status prompt_attn_paged_b8(const va_bf16* q, int n_seqs, int n_tokens, int n_kv_heads, int group,
                               const int32_t* first_row, const int32_t* n_live, const int32_t* lens,
                               const int32_t* table, int max_pages, const void* k_codes, const void* v_codes,
                               const float* k_scale, const float* v_scale, int n_pages, int format, int window,
                               float scale, const float* sink, void* workspace, size_t workspace_bytes, va_bf16* out,
                               float* out_lse, int32_t* dev_status, va_stream stream) {
    using namespace va::paged;
    const size_t need = va_prompt_workspace_bytes(n_seqs, n_tokens, n_kv_heads, group);
    if (need == 0 || !q || !first_row || !n_live || !lens || !table || !workspace || !out) return VA_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || workspace_bytes < need) return VA_INVALID_ARG;
    if (max_pages < 1 || max_pages > 0x7FFFFFFF / kPage || window < 0 || !std::isfinite(scale)) return VA_INVALID_ARG;
    if (format != VA_B8_E4M3 && format != VA_B8_INT8) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, 1, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    pr::Args a = {};
    a.q = q; a.first_row = first_row; a.n_live = n_live; a.lens = lens; a.table = table;
    a.k_codes = static_cast<const uint8_t*>(k_codes); a.v_codes = static_cast<const uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale; a.sink = sink; a.out = out; a.out_lse = out_lse; a.dev_status = dev_status;
    a.scale_log2 = fabsf(scale) * pr::kLog2e; a.flip = scale < 0.0f ? 0x80008000u : 0u;
    a.n_seqs = n_seqs; a.n_rows = n_tokens; a.n_kv = n_kv_heads; a.group = group; a.max_pages = max_pages; a.n_pages = n_pages;
    a.window = window; a.share = 1; a.n_splits = 1;
    a.by_group = pr::Divisor(group); a.by_slots = pr::Divisor(a.share + 1); a.by_rows = pr::Divisor(a.n_rows);
    a.shift = pr::cost_shift((long long)n_kv_heads * (n_seqs + (long long)n_tokens * group / pr::kPairs), max_pages);
    const int sms = va::device_sm_count();
    a.n_ctas = sms > 0 && sms < kMaxCtas ? sms : kMaxCtas;
    pr::place(a, workspace, pr::layout(n_seqs, n_tokens, n_kv_heads, group, false));
    st = launched(format == VA_B8_INT8 ? pr::launch_int8(a, false, (cudaStream_t)stream) : pr::launch_e4m3(a, false, (cudaStream_t)stream));
    if (st != VA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    // (two CTAs an SM, as many as run at a time: with four 4 x 1K prompts took 23.2 us instead of 22.5, with six 24.4.  A call
    // whose rows all fit one unit needs no more than a CTA a row and head)
    const long long pairs = (long long)n_tokens * n_kv_heads * group;
    va::pdl_config(&cfg, attr, dim3((unsigned)(pairs < 2 * a.n_ctas ? pairs : 2 * a.n_ctas)), dim3(pr::kJoinThreads), 0, (cudaStream_t)stream);
    return launched(cudaLaunchKernelEx(&cfg, pr::join_prompt_kernel, a));
}

va_status verify_attn_shared_b8(const va_bf16* q, int n_seqs, int n_rows, int n_kv_heads, int group, int share,
                                const int32_t* n_live, const int32_t* lens, const int32_t* table, int max_pages,
                                const void* k_codes, const void* v_codes, const float* k_scale, const float* v_scale,
                                int n_pages, int format, int window, float scale, const float* sink, void* workspace,
                                size_t workspace_bytes, va_bf16* out, float* out_lse, int32_t* dev_status,
                                va_stream stream) {
    using namespace va::paged;
    const size_t need = va_shared_workspace_bytes(n_seqs, n_rows, n_kv_heads, group);
    if (need == 0 || !q || !n_live || !lens || !table || !workspace || !out) return VA_INVALID_ARG;
    if (share < 0 || (share > 0 && n_seqs % share != 0)) return VA_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || workspace_bytes < need) return VA_INVALID_ARG;
    if (max_pages < 1 || max_pages > 0x7FFFFFFF / kPage || window < 0 || !std::isfinite(scale)) return VA_INVALID_ARG;
    if (format != VA_B8_E4M3 && format != VA_B8_INT8) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, 1, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    if (share == 0) share = n_seqs;
    if (pr::slot_by_slot(n_seqs, n_rows, n_kv_heads, group, share, max_pages, window))
        return verify_attn_paged_b8(q, n_seqs, n_rows, n_kv_heads, group, n_live, lens, table, max_pages, k_codes, v_codes, k_scale,
                                    v_scale, n_pages, format, window, scale, sink, workspace, workspace_bytes, out, out_lse,
                                    dev_status, stream);
    pr::Args a = {};
    a.q = q; a.n_live = n_live; a.lens = lens; a.table = table;
    a.k_codes = static_cast<const uint8_t*>(k_codes); a.v_codes = static_cast<const uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale; a.sink = sink; a.out = out; a.out_lse = out_lse; a.dev_status = dev_status;
    a.scale_log2 = fabsf(scale) * pr::kLog2e; a.flip = scale < 0.0f ? 0x80008000u : 0u;
    a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_kv = n_kv_heads; a.group = group; a.max_pages = max_pages; a.n_pages = n_pages;
    a.window = window; a.share = share;
    a.by_group = pr::Divisor(group); a.by_slots = pr::Divisor(a.share + 1); a.by_rows = pr::Divisor(a.n_rows);
    const int splits = (max_pages + pr::kCommonPages - 1) / pr::kCommonPages;
    a.n_splits = splits < pr::kSplits ? splits : pr::kSplits;
    a.shift = pr::cost_shift((long long)n_kv_heads * (2 * n_seqs + (long long)n_seqs * n_rows * group / pr::kPairs), max_pages);
    const int sms = va::device_sm_count();
    a.n_ctas = sms > 0 && sms < kMaxCtas ? sms : kMaxCtas;
    pr::place(a, workspace, pr::layout(n_seqs, n_rows, n_kv_heads, group, true));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)(n_seqs / a.share), (unsigned)a.n_splits), dim3(pr::kCommonThreads), 0, (cudaStream_t)stream);
    st = launched(cudaLaunchKernelEx(&cfg, pr::common_kernel, a));
    if (st != VA_OK) return st;
    st = launched(format == VA_B8_INT8 ? pr::launch_int8(a, true, (cudaStream_t)stream) : pr::launch_e4m3(a, true, (cudaStream_t)stream));
    if (st != VA_OK) return st;
    // a row and head a CTA where there are two an SM at most, else a warp
    const long long total = (long long)n_seqs * n_rows * n_kv_heads * group;
    const long long ctas = total <= 2 * a.n_ctas ? total : (total + pr::kJoinWarps - 1) / pr::kJoinWarps;
    va::pdl_config(&cfg, attr, dim3((unsigned)ctas), dim3(pr::kJoinThreads), 0, (cudaStream_t)stream);
    return launched(cudaLaunchKernelEx(&cfg, pr::join_shared_kernel, a));
}

}  // extern "C"
