// What the two split kernels of verify_attn_paged_b8 (paged_attn.cuh, paged_attn_tc.cuh) and its joining kernel
// share: the arguments, the deal of the batch's tiles over the CTAs, the walk over a CTA's segments, the end of a row.
//
// A sequence's visible pages, times its KV heads, are its tiles (64 keys of one head); all tiles of the batch in
// (sequence, head, page) order are dealt to one CTA an SM by cost, whatever the lengths.  A run of tiles of one
// (sequence, head) in a CTA is a segment.  A segment that covers its head writes the output itself; the others (at
// most the first and the last of a CTA) leave partial sums that a second launch joins.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace va {
namespace paged {

constexpr int kMaxCtas = 160;                 // CTAs of one call (one an SM)
constexpr int kMaxCols = VA_MAX_ROWS * VA_PAGED_MAX_GROUP;   // 64 (row, query head) pairs of a KV head
constexpr int kTileBytes = 2 * kHeadBytes;    // K and V codes of a tile
constexpr uint64_t kWaitNs = 1000000000ull;   // a wait gives up after a second (VA_DEV_TIMEOUT)
constexpr float kShift = 6.0f;                // p = 2^(t - m + kShift)
constexpr float kLazy = 8.0f;                 // m is raised when a score passes it by this much
constexpr int kFewPairs = 16;                 // pairs that paged_attn.cuh takes; paged_attn_tc.cuh more
constexpr float kNoScore = -3.0e38f;          // m before the first score (any score passes it)

// Workspace: partial sums of 2 segments a CTA, [2 kMaxCtas][kMaxCols][128] floats, then their (m, l).
constexpr size_t kPartFloats = (size_t)2 * kMaxCtas * kMaxCols * kD;
constexpr size_t kWorkspaceBytes = sizeof(float) * (kPartFloats + (size_t)2 * kMaxCtas * kMaxCols * 2);

struct AttnPagedArgs {
    const uint16_t* q;
    const int32_t *n_live, *lens, *table;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const float* sink;
    float* part_o;
    float2* part_ml;
    uint16_t* out;
    float* out_lse;
    int32_t* dev_status;
    float scale_log2;                         // scale x log2 e
    int n_seqs, n_rows, n_kv, group, max_pages, n_pages, window, n_ctas;
};

// The first position that a row of a sequence sees, or less.
__device__ __forceinline__ int seen_from(int len, int live, int window) { return window > 0 ? len - live - window + 1 : 0; }

// The visible pages of a sequence: [first, first + n).
struct Span {
    int first, n;
};
__device__ __forceinline__ Span span_of(int len, int live, int window) {
    Span s;
    s.first = max(0, seen_from(len, live, window)) / kPage;
    s.n = live > 0 ? (len + kPage - 1) / kPage - s.first : 0;
    return s;
}

// The deal.  A segment costs a CTA about as much as kSegCost tiles besides its tiles (its q, its joining, code that is
// not in the instruction cache), so the tiles are dealt by cost: the tiles of a (sequence, head) of n pages lie at the
// costs s + kSegCost .. s + kSegCost + n - 1, the next head's at s + kSegCost + n on, and CTA c of C takes the tiles
// whose cost is in [c W / C, (c + 1) W / C), W the sum.  Measured, decode of 64 ragged sequences of 1 to 16K, 8 heads:
// 75.4 us at 2, 68.2 at 4, 62.4 at 8, 58.7 at 10, 59.7 at 13; a window of 4,096 over 32 sequences: 42.6, 37.1, 36.6,
// 37.1, 38.6.
constexpr int kSegCost = 10;
__device__ __forceinline__ long long cta_begin(int c, int n, long long total) {
    return total < (1ll << 24) ? (long long)((unsigned)c * (unsigned)total / (unsigned)n) : (long long)c * total / n;
}

// What an unnormalised output row sum 2^(t - m) v is multiplied by, and its log-sum-exp: l is the sum of 2^(t - m),
// the sink joins the denominator.
struct Finish {
    float by, lse;
};
__device__ __forceinline__ Finish finish(float m, float l, const float* sink, int head) {
    Finish f;
    const float s2 = sink ? __ldg(sink + head) * 1.4426950408889634f : -INFINITY;
    const float seen = l == 0.0f ? -INFINITY : m + log2f(l);
    const float top = fmaxf(seen, s2);
    const float all = top == -INFINITY ? -INFINITY : top + log2f(exp2f(seen - top) + exp2f(s2 - top));
    f.by = l == 0.0f ? 0.0f : (l != l ? l : exp2f(seen - all) / l);
    f.lse = (l != l ? l : all) * 0.6931471805599453f;
    return f;
}

__device__ __forceinline__ void store_row(uint16_t* dst, const float4& o) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A wait that the warp makes as one: every lane leaves it with the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int& status) {
    const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort, kWaitNs));
    if (!ok) {
        if (!*abort) status |= VA_DEV_TIMEOUT;
        __syncwarp();
        *abort = 1;
    }
    return ok;
}

// The deal, in shared memory: tiles before each sequence, sequences with tiles before it, lengths and live rows; and
// the row and query head of each of a KV head's pairs.
struct Plan {
    long long pre[VA_PAGED_MAX_SEQS + 1];
    unsigned long long sums[32];
    int len[VA_PAGED_MAX_SEQS];
    unsigned short some[VA_PAGED_MAX_SEQS + 2];
    signed char live[VA_PAGED_MAX_SEQS];
    unsigned char col_row[kMaxCols], col_head[kMaxCols];
};

// What a CTA has of it: tiles c0 .. c0 + n - 1, the first of them tile t of head h of sequence b.
struct Share {
    long long c0;
    int n, b, h, t, n_ctas;
};

// The last sequence that begins at or before x, in tiles (seg = 0) or in costs (seg = kSegCost x heads).
__device__ __forceinline__ int find_seq(const Plan& p, int n_seqs, long long x, int seg) {
    int lo = 0, hi = n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.pre[mid] + seg * (int)p.some[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Every thread of a CTA of kThreads calls it, after the launch dependency has resolved; two block barriers.
template <int kThreads>
__device__ __forceinline__ Share make_plan(Plan& p, const AttnPagedArgs& a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = (VA_PAGED_MAX_SEQS + kThreads - 1) / kThreads;   // sequences per thread
    if (tid < kMaxCols) {
        p.col_row[tid] = (unsigned char)(tid / a.group);
        p.col_head[tid] = (unsigned char)(tid % a.group);
    }
    // per thread: tiles in the low 48 bits, sequences that have any above (at most 1,024)
    unsigned long long mine[kPer], sum = 0;
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    int status = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        mine[i] = 0;
        if (i < per && b < a.n_seqs) {
            const Seq s = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
            status |= s.status;
            p.len[b] = s.len;
            p.live[b] = (signed char)s.live;
            const int n = span_of(s.len, s.live, a.window).n;
            mine[i] = (unsigned long long)n * a.n_kv + (n > 0 ? 1ull << 48 : 0ull);
            sum += mine[i];
        }
    }
    unsigned long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) p.sums[warp] = upto;
    __syncthreads();
    unsigned long long before = upto - sum;
    for (int w = 0; w < warp; ++w) before += p.sums[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.n_seqs) {
            p.pre[b] = (long long)(before & 0xFFFFFFFFFFFFull);
            p.some[b] = (unsigned short)(before >> 48);
            before += mine[i];
            if (b == a.n_seqs - 1) {
                p.pre[a.n_seqs] = (long long)(before & 0xFFFFFFFFFFFFull);
                p.some[a.n_seqs] = (unsigned short)(before >> 48);
            }
        }
    }
    if (status && a.dev_status && blockIdx.x == 0) atomicOr(a.dev_status, status);
    __syncthreads();
    // where this CTA's tiles begin (even lanes) and the next one's (odd lanes)
    const long long total = p.pre[a.n_seqs];
    const int seg_cost = kSegCost * a.n_kv;
    const long long cost = total + seg_cost * (int)p.some[a.n_seqs];
    Share s;
    s.n_ctas = (int)min((long long)a.n_ctas, total);
    s.c0 = total;
    s.b = s.h = s.t = s.n = 0;
    if ((int)blockIdx.x >= s.n_ctas) return s;
    const long long y = cta_begin(blockIdx.x + (lane & 1), s.n_ctas, cost);
    if (y < cost) {
        s.b = find_seq(p, a.n_seqs, y, seg_cost);
        const unsigned rest = (unsigned)(y - p.pre[s.b] - seg_cost * (int)p.some[s.b]);
        const unsigned n = (unsigned)span_of(p.len[s.b], p.live[s.b], a.window).n, per_head = n + kSegCost;
        s.h = (int)(rest / per_head);
        s.t = max((int)(rest % per_head) - kSegCost, 0);
        s.c0 = p.pre[s.b] + (long long)s.h * n + s.t;
    }
    const long long end = __shfl_sync(0xffffffffu, s.c0, 1);
    s.c0 = __shfl_sync(0xffffffffu, s.c0, 0);
    s.b = __shfl_sync(0xffffffffu, s.b, 0);
    s.h = __shfl_sync(0xffffffffu, s.h, 0);
    s.t = __shfl_sync(0xffffffffu, s.t, 0);
    s.n = (int)(end - s.c0);                     // none where the CTA's costs are all a segment's own
    return s;
}

// The pool row (page x heads + head) of tile i of a CTA's share, or -1 (and a status bit) if it is no page.
__device__ __forceinline__ int tile_row(const Plan& p, const AttnPagedArgs& a, long long x, int& status) {
    const int b = find_seq(p, a.n_seqs, x, 0);
    const Span sp = span_of(p.len[b], p.live[b], a.window);
    const unsigned within = (unsigned)(x - p.pre[b]);
    const int h = (int)(within / (unsigned)sp.n), t = sp.first + (int)(within % (unsigned)sp.n);
    const int page = __ldcg(a.table + (size_t)b * a.max_pages + t);
    if (page >= 0 && page < a.n_pages) return page * a.n_kv + h;
    status |= VA_DEV_BAD_PAGE;
    return -1;
}

// The segments of a share, in order.
struct Walk {
    int b, h, len, live;     // of the segment
    int page0;               // its first page's index in the sequence
    int begin, end;          // its tiles, counted from the CTA's first
    int seg;
    bool whole;              // it covers its head
    int b_next, h_next, t_next;
    __device__ __forceinline__ explicit Walk(const Share& s) {
        seg = -1;
        begin = end = 0;
        b_next = s.b;
        h_next = s.h;
        t_next = s.t;
    }
    __device__ __forceinline__ bool next(const Plan& p, const AttnPagedArgs& a, int n_tiles) {
        if (end >= n_tiles) return false;
        begin = end;
        b = b_next;
        h = h_next;
        ++seg;
        len = p.len[b];
        live = p.live[b];
        const Span sp = span_of(len, live, a.window);
        page0 = sp.first + t_next;
        const int n = min(n_tiles - begin, sp.n - t_next);
        whole = n == sp.n;
        end += n;
        t_next = 0;
        if (++h_next == a.n_kv) {
            h_next = 0;
            do ++b_next;
            while (b_next < a.n_seqs && p.pre[b_next + 1] == p.pre[b_next]);
        }
        return true;
    }
};

}  // namespace paged
}  // namespace va
