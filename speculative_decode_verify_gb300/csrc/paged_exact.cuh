// The end of a CTA of verify_attn_paged_b8's split kernels whose V scales lie too far apart for weights in f16.
//
// The split kernels hold weights w = p s in f16, p = 2^(t - m + 6) and s a block's V scale relative to the largest so far.
// A scale more than 2^10 below that brings the weights of its keys, at 2^6 units by themselves, to where f16 begins to
// lose digits: at 2^-5, where n others that are rounded to 2^-25 of a unit cost them n 2^-20, and from a ratio of 2^31 on
// nothing is left, though these keys may carry all the weight.  And at the other end the sums of 2^6 to 2^14 v pass fp32's
// range where scales pass 2^104.  A CTA that has met scales that far apart (0 aside) or above 2^90 computes its segments
// with such scales again, here: in fp32, from the definition, over what the segment has left.
//   Eight warps share a segment's pages and take its (row, query head) pairs one after the other; a lane has two keys'
// scores and four dimensions' sums.  Caches hardly hold such scales, so this is short rather than fast.  With one block of
// 2^-20 in each sequence, decode of 64 ragged sequences of 1 to 16K takes 1.0 ms (59 us without), 48 pairs of one
// sequence of 192K 1.1 ms (37 us).  Being there costs the ordinary calls 0.1 to 0.7 us; in the joining kernel, behind its
// ordinary end, it cost each 1 to 1.5 us, and code unrolled further, or not marked as unlikely, another 0.7 us of the
// windows.
#pragma once

#include "paged_plan.cuh"

namespace va {
namespace paged {

constexpr float kFar = 1024.0f;
constexpr float kHuge = 1.2379400e27f;      // 2^90
constexpr int kExactWarps = 8;

struct ExactSmem {
    float4 acc[kExactWarps][32];
    float2 ml[kExactWarps];
    float q[kD];
};

// Whether the V scales of pages x0 .. x1 - 1 that some row sees lie far apart or high.  Half of kFar and kHuge: at least as
// soon as a split kernel, whose unit is up to twice the largest scale.  Every warp looks at all pages.
__device__ __forceinline__ bool scales_far_apart(const AttnPagedArgs& a, const Walk& w, int x0, int x1) {
    const int lane = threadIdx.x & 31, from = seen_from(w.len, w.live, a.window);
    uint32_t lowest = 0x7F800000u, highest = 0u;      // (positive floats order like their bits)
    for (int x = x0 + lane; x < x1; x += 32) {
        const int page = __ldcg(a.table + (size_t)w.b * a.max_pages + x);
        if (page < 0 || page >= a.n_pages) continue;
#pragma unroll 1
        for (int k = 0; k < kBlocks; ++k) {
            const float s = __ldcg(a.v_scale + ((size_t)page * a.n_kv + w.h) * kBlocks + k);
            const int at = x * kPage + k * kBlock;
            if (at < w.len && at + kBlock > from && s > 0.0f) {
                lowest = min(lowest, __float_as_uint(s));
                highest = max(highest, __float_as_uint(s));
            }
        }
    }
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);
    return __uint_as_float(highest) > fminf(kFar / 2 * __uint_as_float(lowest), kHuge / 2);
}

// Pair `col` over pages x0 .. x1 - 1.
template <bool kInt8>
__device__ __forceinline__ void exact_pair(const AttnPagedArgs& a, const Plan& plan, const Walk& seg, int x0, int x1, int col,
                                           ExactSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = seg.h * a.group + plan.col_head[col];
    const size_t row = ((size_t)seg.b * a.n_rows + plan.col_row[col]) * (a.n_kv * a.group) + head;
    const int p = seg.len - seg.live + plan.col_row[col], lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
    if (tid < kD) sm.q[tid] = __uint_as_float((uint32_t)a.q[row * kD + tid] << 16);
    ptx::named_bar_sync(1, 32 * kExactWarps);
    float top = -INFINITY, sum = 0.0f;      // sum: this lane's keys'
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = max(x0, lo / kPage) + warp; x < min(x1, p / kPage + 1); x += kExactWarps) {
        const int page = __ldcg(a.table + (size_t)seg.b * a.max_pages + x);
        if (page < 0 || page >= a.n_pages) continue;
        const size_t at = (size_t)page * a.n_kv + seg.h;
        const uint8_t *k = a.k_codes + at * kHeadBytes, *v = a.v_codes + at * kHeadBytes;
        const int first = max(lo - x * kPage, 0), last = min(p - x * kPage, kPage - 1);      // the keys that the row sees
        float t[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int key = lane + 32 * e;
            float dot = 0.0f;
#pragma unroll 2
            for (int c = 0; c < kD / 16; ++c) {
                const uint4 w = reinterpret_cast<const uint4*>(k + key * kD)[c];
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float c4[4];
                    decode4<kInt8>(words[i], c4);
#pragma unroll
                    for (int d = 0; d < 4; ++d) dot = fmaf(c4[d], sm.q[16 * c + 4 * i + d], dot);
                }
            }
            t[e] = key < first || key > last ? -INFINITY : dot * (a.k_scale[at * kBlocks + key / kBlock] * a.scale_log2);
        }
        float now = fmaxf(t[0], t[1]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
        now = fmaxf(now, top);
        const float ref = now == -INFINITY ? 0.0f : now, by = top == -INFINITY ? 1.0f : exp2f(top - ref);
        top = now;
        acc.x *= by;
        acc.y *= by;
        acc.z *= by;
        acc.w *= by;
        const float w0 = exp2f(t[0] - ref), w1 = exp2f(t[1] - ref);
        sum = sum * by + (w0 + w1);
        // (of keys that the row does not see: weight 0, and codes that may be NaN)
#pragma unroll 1
        for (int block = first / kBlock; block <= last / kBlock; ++block) {
            const float s = a.v_scale[at * kBlocks + block];
#pragma unroll 8
            for (int i = 0; i < kBlock; ++i) {
                const int key = block * kBlock + i;
                const float w = s * __shfl_sync(0xffffffffu, block < 2 ? w0 : w1, key & 31);
                const uint32_t word = reinterpret_cast<const uint32_t*>(v + key * kD)[lane];
                float x4[4];
                decode4<kInt8>(key < first || key > last ? 0u : word, x4);
                acc.x = fmaf(w, x4[0], acc.x);
                acc.y = fmaf(w, x4[1], acc.y);
                acc.z = fmaf(w, x4[2], acc.z);
                acc.w = fmaf(w, x4[3], acc.w);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sm.acc[warp][lane] = acc;
    if (lane == 0) sm.ml[warp] = make_float2(top, sum);
    ptx::named_bar_sync(1, 32 * kExactWarps);
    if (warp != 0) return;                  // (the others' next words wait for warp 0 at the next pair's barrier)
    top = -INFINITY;
    for (int w = 0; w < kExactWarps; ++w) top = fmaxf(top, sm.ml[w].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.0f;
#pragma unroll 1
    for (int w = 0; w < kExactWarps; ++w) {
        const float2 one = sm.ml[w];
        const float f = one.x == -INFINITY ? (one.y != one.y ? one.y : 0.0f) : exp2f(one.x - top);
        const float4 v = sm.acc[w][lane];
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
        sum = fmaf(f, one.y, sum);
    }
    if (seg.whole) {
        const Finish f = finish(top, sum, a.sink, head);
        store_row(a.out + row * kD + 4 * lane, make_float4(acc.x * f.by, acc.y * f.by, acc.z * f.by, acc.w * f.by));
        if (lane == 0 && a.out_lse) a.out_lse[row] = f.lse;
    } else {
        const size_t part = (size_t)(2 * blockIdx.x + (seg.begin == 0 ? 0 : 1)) * kMaxCols + col;
        reinterpret_cast<float4*>(a.part_o + part * kD)[lane] = acc;
        if (lane == 0) a.part_ml[part] = make_float2(top, sum);
    }
}

// The segments of a CTA's share whose scales lie far apart.  Warps 0 .. kExactWarps - 1 call it, once what the CTA has
// written is ordered before it (a barrier).
template <bool kInt8>
__device__ __forceinline__ void exact_segments(const AttnPagedArgs& a, const Plan& plan, const Share& share, ExactSmem& sm) {
    Walk seg(share);
    while (seg.next(plan, a, share.n)) {
        const int x0 = seg.page0, x1 = seg.page0 + seg.end - seg.begin;
        if (!scales_far_apart(a, seg, x0, x1)) continue;
#pragma unroll 1
        for (int col = 0; col < seg.live * a.group; ++col) exact_pair<kInt8>(a, plan, seg, x0, x1, col, sm);
    }
}

}  // namespace paged
}  // namespace va
