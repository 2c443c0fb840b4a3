// kv_page_append_rope_b8: queries and keys rotated by their positions, keys and values coded into the pages.
//
// The unit of work is the rows of 16 positions of one sequence (one scale's worth), or a part of their heads where a call has
// few such blocks.  A CTA brings their cosines and sines into shared memory once, and its warps share out the heads: for
// keys and values a warp codes one head's block (half a warp a row, eight rows a lane in fp32 registers), for queries half a
// warp takes eight heads of a row at a time, the next eight on their way.  A lane's eight elements of a row are four whole
// pairs, two times four elements that lie rot_dim / 2 apart or next to each other, so that no lane asks another.
//
// Bound by memory: 16K tokens of 48 + 2 x 8 heads take 94 us (5.4 TB/s of what has to be read and written; a copy of as much
// 75), with 216 to 240 bytes of spills at 128 registers, two CTAs an SM.  Calls of single tokens are bound by their launch and
// the chain of loads (lengths, table, rows): 7 us for 64 of them.
#include <cuda_bf16.h>

#include "paged_code.cuh"
#include "tc_ptx.cuh"

#include "kv_prompts.h"

namespace va {
namespace paged {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeQ = 8;                // rows of a query head that a half warp has in flight

struct RopeArgs {
    const uint16_t *q, *k_new, *v_new;
    const int32_t *first_row, *n_live, *lens, *table;
    const float* cos_sin;
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    uint16_t* q_out;
    int32_t* dev_status;
    int n_seqs, n_tokens, n_kv, heads, max_pages, n_positions, rot, n_pages;
    int parts;                   // CTAs that share a block's heads
};

struct RopeSeq {
    int len, live, first, status;
};
__device__ __forceinline__ RopeSeq rope_seq(const RopeArgs& a, int b) {
    const Seq s = load_seq(a.lens, a.n_live, b, a.n_tokens, a.max_pages);
    RopeSeq r;
    r.len = s.len;
    r.live = s.live;
    r.status = s.status;
    r.first = __ldcg(a.first_row + b);
    if (r.live > 0 && (r.first < 0 || r.first > a.n_tokens - r.live)) r.status |= VA_DEV_BAD_COUNT;
    if (r.len > a.n_positions && r.live > 0) r.status |= VA_DEV_BEYOND_TABLE;
    if (r.status) r.len = r.live = 0;
    return r;
}
__device__ __forceinline__ int rope_blocks(const RopeSeq& s) {
    return s.live > 0 ? (s.len - 1) / kBlock - (s.len - s.live) / kBlock + 1 : 0;
}

// A lane's place in rows of 128: elements o0 .. o0 + 3 and o1 .. o1 + 3, which are pairs 4 li .. 4 li + 3 where `turns`.
struct Lane {
    int o0, o1;
    bool turns;
    const float *c, *s;          // the pairs' cosines and sines in row 0 of the table in shared memory
    __device__ __forceinline__ Lane(int rot, bool interleaved, bool rotate, const float* table) {
        const int li = threadIdx.x & 15;
        turns = rotate && li < rot / 8;
        o0 = 8 * li;             // (of the dimensions that pass a lane has eight next to each other: from rot on as well)
        o1 = o0 + 4;
        if (turns && !interleaved) {
            o0 = 4 * li;
            o1 = rot / 2 + 4 * li;
        }
        c = table + 4 * li;
        s = c + rot / 2;
    }
};
__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ float2 times(float2 a, float2 b) { return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)); }

// The lane's eight elements, rotated where they turn; c and s are those of its pairs.
template <bool kInterleaved>
__device__ __forceinline__ void rotate8(const uint2& u, const uint2& v, bool turns, const float4& c, const float4& s, float (&x)[8]) {
    const float2 p[4] = {pair_of(u.x), pair_of(u.y), pair_of(v.x), pair_of(v.y)};
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = p[i].x;
        x[2 * i + 1] = p[i].y;
    }
    if (!turns) return;
    if (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = times(p[i], make_float2(cc[i], cc[i])), b = times(p[i], make_float2(ss[i], ss[i]));
            x[2 * i] = __fsub_rn(a.x, b.y);
            x[2 * i + 1] = __fadd_rn(a.y, b.x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[i], b = x[4 + i];
            x[i] = __fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i]));
            x[4 + i] = __fadd_rn(__fmul_rn(b, cc[i]), __fmul_rn(a, ss[i]));
        }
    }
}

// What few blocks need is out of line: the kernel's code is fetched anew by each launch, and inlined over and over these made
// it 180 KB.  Quotients that need a division, or older codes coded again.
template <bool kInt8>
__device__ __noinline__ uint2 divide8(float4 a, float4 b, float s) {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return code8<kInt8, true>(x, s, 0.0f, true);
}
template <bool kInt8>
__device__ __noinline__ uint2 again8(uint2 c, float was, float s) {
    float a[4], b[4], x[8];
    decode4<kInt8>(c.x, a);
    decode4<kInt8>(c.y, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = __fmul_rn(a[e], was);
        x[4 + e] = __fmul_rn(b[e], was);
    }
    return code8<kInt8, true>(x, s, __frcp_rn(s), !(s > 8.3e-25f));
}

// One head's block of keys or values: the rows lo .. hi - 1 of the 16 positions from p0 on are new.
template <bool kInt8, bool kInterleaved>
__device__ __forceinline__ int code_block(const uint16_t* src, int stride, const Lane& at, int lo, int hi, int p0, uint8_t* codes,
                                          float* scale) {
    const int lane = threadIdx.x & 31, half = lane >> 4;
    uint2 u[8], v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int p = p0 + 2 * r + half;
        u[r] = v[r] = make_uint2(0u, 0u);
        if (p >= lo && p < hi) {
            const uint16_t* row = src + (size_t)(p - lo) * stride;
            u[r] = __ldcs(reinterpret_cast<const uint2*>(row + at.o0));
            v[r] = __ldcs(reinterpret_cast<const uint2*>(row + at.o1));
        }
    }
    const bool older = p0 < lo;
    const float was = older ? __ldcg(scale) : 0.0f;
    float x[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        // (the table's rows of positions that are not new hold anything: their elements are not looked at)
        const float* c = at.c + (2 * r + half) * kD;
        const float* s = at.s + (2 * r + half) * kD;
        rotate8<kInterleaved>(u[r], v[r], at.turns, *reinterpret_cast<const float4*>(c), *reinterpret_cast<const float4*>(s), x[r]);
        const int p = p0 + 2 * r + half;
        uint32_t here = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) here = max(here, __float_as_uint(x[r][e]) & 0x7FFFFFFFu);
        if (p >= lo && p < hi) top = max(top, here);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const bool special = top >= 0x7F800000u;
    if (special) {
        // an infinity or NaN somewhere: the largest finite one instead, and NaN becomes 0
        top = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int p = p0 + 2 * r + half;
            const bool in = p >= lo && p < hi;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = __float_as_uint(x[r][e]) & 0x7FFFFFFFu;
                if (m > 0x7F800000u) x[r][e] = 0.0f;
                if (in && m < 0x7F800000u) top = max(top, m);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
    }
    const float fresh = __fdiv_rn(__uint_as_float(top), top_code(kInt8));
    const float s = older ? fmaxf(fresh, was) : fresh;
    const bool careful = special || !(s > 8.3e-25f);      // as in paged_append.cu
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int p = p0 + 2 * r + half;
        if (p < lo || p >= hi) continue;
        const uint2 w = careful ? divide8<kInt8>(make_float4(x[r][0], x[r][1], x[r][2], x[r][3]), make_float4(x[r][4], x[r][5], x[r][6], x[r][7]), s)
                                : code8<kInt8, true>(x[r], s, inv, false);
        *reinterpret_cast<uint32_t*>(codes + (2 * r + half) * kD + at.o0) = w.x;
        *reinterpret_cast<uint32_t*>(codes + (2 * r + half) * kD + at.o1) = w.y;
    }
    if (older && s > was) {
        // the older rows' codes, all on their way at once
        uint2 held[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            held[r] = make_uint2(0u, 0u);
            if (p0 + 2 * r + half < lo) held[r] = *reinterpret_cast<const uint2*>(codes + (2 * r + half) * kD + 8 * (lane & 15));
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (p0 + 2 * r + half < lo) *reinterpret_cast<uint2*>(codes + (2 * r + half) * kD + 8 * (lane & 15)) = again8<kInt8>(held[r], was, s);
    }
    __syncwarp();
    if (lane == 0) *scale = s;
    return special ? VA_DEV_NONFINITE : 0;
}

template <bool kInt8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_append_kernel(const RopeArgs a) {
    __shared__ alignas(16) float cs[kBlock * kD];
    __shared__ int before[VA_PAGED_MAX_SEQS + 1];
    __shared__ int sums[kRopeWarps];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = lane >> 4;
    int status = 0;
    // blocks before each sequence
    constexpr int kPer = VA_PAGED_MAX_SEQS / kRopeThreads;
    const int per = (a.n_seqs + kRopeThreads - 1) / kRopeThreads;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        mine[i] = 0;
        if (i < per && b < a.n_seqs) {
            const RopeSeq s = rope_seq(a, b);
            status |= s.status;
            mine[i] = rope_blocks(s);
            sum += mine[i];
        }
    }
    if (blockIdx.x != 0) status = 0;     // one CTA tells
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int at = upto - sum;
    for (int w = 0; w < warp; ++w) at += sums[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.n_seqs) {
            before[b] = at;
            at += mine[i];
            if (b == a.n_seqs - 1) before[a.n_seqs] = at;
        }
    }
    __syncthreads();
    const int total = before[a.n_seqs], rot = a.rot;
    for (long long work = blockIdx.x; work < (long long)total * a.parts; work += gridDim.x) {
        const int unit = (int)(work / a.parts), part = (int)(work % a.parts);
        int b = 0, end = a.n_seqs;
        while (end - b > 1) {
            const int mid = (b + end) >> 1;
            if (before[mid] <= unit) b = mid;
            else end = mid;
        }
        const RopeSeq s = rope_seq(a, b);
        const int start = s.len - s.live, block = start / kBlock + unit - before[b], p0 = block * kBlock;
        const int lo = max(p0, start), hi = min(s.len - p0, kBlock) + p0;
        const int page = __ldcg(a.table + (size_t)b * a.max_pages + block / kBlocks);
        __syncthreads();                                    // the table of the work before has been used
        for (int i = tid; i < (hi - lo) * (rot >> 2); i += kRopeThreads) {
            const int r = i / (rot >> 2), c = i % (rot >> 2);
            *reinterpret_cast<float4*>(cs + (lo - p0 + r) * kD + 4 * c) =
                __ldg(reinterpret_cast<const float4*>(a.cos_sin + (size_t)(lo + r) * rot) + c);
        }
        const size_t row0 = (size_t)s.first + (lo - start);    // of the packed rows
        // this part's warps share out the heads' blocks of keys and of values, then the rows of query heads, sixteen at a time
        const bool page_ok = page >= 0 && page < a.n_pages;
        if (!page_ok) status |= VA_DEV_BAD_PAGE;
        const int n_code = page_ok ? 2 * a.n_kv : 0, step = kRopeWarps * a.parts, me = part * kRopeWarps + warp;
        const int per_row = (a.heads + 2 * kRopeQ - 1) / (2 * kRopeQ), n_items = a.q ? (hi - lo) * per_row : 0;
        __syncthreads();
#pragma unroll 1
        for (int h2 = me; h2 < n_code; h2 += step) {
            const int h = h2 >> 1;
            const bool is_v = h2 & 1;
            const size_t head = (size_t)page * a.n_kv + h, of = block % kBlocks;
            const Lane at(rot, kInterleaved, !is_v, cs);
            status |= code_block<kInt8, kInterleaved>((is_v ? a.v_new : a.k_new) + (row0 * a.n_kv + h) * kD, a.n_kv * kD, at, lo, hi, p0,
                                                      (is_v ? a.v_codes : a.k_codes) + head * kHeadBytes + of * kBlock * kD,
                                                      (is_v ? a.v_scale : a.k_scale) + head * kBlocks + of);
        }
        // item: (row, heads 16 i .. 16 i + 15), every other one half a warp's
        const Lane at(rot, kInterleaved, true, cs);
        int item = (me + step - n_code % step) % step;         // (the warps that code come last)
        uint2 u[kRopeQ], v[kRopeQ];
        auto load = [&](int i) {
            const int r = i / per_row, h0 = (i - r * per_row) * 2 * kRopeQ + half;
            const uint16_t* src = a.q + ((row0 + r) * a.heads + h0) * kD;
#pragma unroll
            for (int k = 0; k < kRopeQ; ++k) {
                u[k] = v[k] = make_uint2(0u, 0u);
                if (i < n_items && h0 + 2 * k < a.heads) {
                    u[k] = __ldcs(reinterpret_cast<const uint2*>(src + 2 * k * kD + at.o0));
                    v[k] = __ldcs(reinterpret_cast<const uint2*>(src + 2 * k * kD + at.o1));
                }
            }
        };
        load(item);
#pragma unroll 1
        for (; item < n_items; item += step) {
            const int r = item / per_row, h0 = (item - r * per_row) * 2 * kRopeQ + half;
            uint16_t* dst = a.q_out + ((row0 + r) * a.heads + h0) * kD;
            const float4 c = *reinterpret_cast<const float4*>(at.c + (lo - p0 + r) * kD), s = *reinterpret_cast<const float4*>(at.s + (lo - p0 + r) * kD);
            uint2 y[kRopeQ], z[kRopeQ];
#pragma unroll
            for (int k = 0; k < kRopeQ; ++k) {
                y[k] = u[k];
                z[k] = v[k];
            }
            load(item + step);
#pragma unroll
            for (int k = 0; k < kRopeQ; ++k) {
                float x[8];
                rotate8<kInterleaved>(y[k], z[k], at.turns, c, s, x);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 f = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                    w[e] = *reinterpret_cast<const uint32_t*>(&f);
                }
                if (h0 + 2 * k < a.heads) {
                    __stcs(reinterpret_cast<uint2*>(dst + 2 * k * kD + at.o0), make_uint2(w[0], w[1]));
                    __stcs(reinterpret_cast<uint2*>(dst + 2 * k * kD + at.o1), make_uint2(w[2], w[3]));
                }
            }
        }
    }
    status = __reduce_or_sync(0xffffffffu, status);
    if (status && a.dev_status && lane == 0) atomicOr(a.dev_status, status);
}

}  // namespace paged
}  // namespace va

extern "C" va_status kv_page_append_rope_b8(const va_bf16* q, const va_bf16* k_new, const va_bf16* v_new, int n_seqs,
                                            int n_tokens, int n_kv_heads, int group, const int32_t* first_row,
                                            const int32_t* n_live, const int32_t* lens, const int32_t* table,
                                            int max_pages, const float* cos_sin, int n_positions, int rot_dim,
                                            int interleaved, void* k_codes, void* v_codes, float* k_scale,
                                            float* v_scale, int n_pages, int format, va_bf16* q_out,
                                            int32_t* dev_status, va_stream stream) {
    using namespace va::paged;
    if (!k_new || !v_new || !first_row || !n_live || !lens || !table || !cos_sin || !q != !q_out) return VA_INVALID_ARG;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(cos_sin))
        return VA_INVALID_ARG;
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || n_tokens < 1 || n_tokens > VA_MAX_TOKENS || group < 1 ||
        group > VA_PAGED_MAX_GROUP || n_positions < 1)
        return VA_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > va::kD || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1)) return VA_INVALID_ARG;
    if (max_pages < 1 || max_pages > 0x7FFFFFFF / kPage) return VA_INVALID_ARG;
    if (format != VA_B8_E4M3 && format != VA_B8_INT8) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, 1, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    RopeArgs a;
    a.q = q; a.k_new = k_new; a.v_new = v_new;
    a.first_row = first_row; a.n_live = n_live; a.lens = lens; a.table = table; a.cos_sin = cos_sin;
    a.k_codes = static_cast<uint8_t*>(k_codes); a.v_codes = static_cast<uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.q_out = q_out; a.dev_status = dev_status;
    a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.n_kv = n_kv_heads; a.heads = n_kv_heads * group;
    a.max_pages = max_pages; a.n_positions = n_positions; a.rot = rot_dim; a.n_pages = n_pages;
    // most blocks of rows that there can be: each sequence begins and ends one that it does not fill
    const int sms = va::device_sm_count() > 0 ? va::device_sm_count() : 152;
    const long long most = (long long)n_tokens / kBlock + 2ll * (n_seqs < n_tokens ? n_seqs : n_tokens);
    const int rows = (n_tokens + n_seqs - 1) / n_seqs < kBlock ? (n_tokens + n_seqs - 1) / n_seqs : kBlock;      // of a block, about
    const int items = 2 * n_kv_heads + (q ? rows * ((a.heads + 2 * kRopeQ - 1) / (2 * kRopeQ)) : 0), useful = (items + kRopeWarps - 1) / kRopeWarps;
    // two CTAs an SM; parts for several works a CTA, or at least a work each
    const int wave = 2 * sms;
    const long long parts = (4ll * wave + most - 1) / most;
    a.parts = (int)(parts < useful ? parts : useful);
    const long long works = most * a.parts;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)(works < wave ? works : wave)), dim3(kRopeThreads), 0, (cudaStream_t)stream);
    cudaError_t e;
    if (format == VA_B8_INT8)
        e = interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<true, true>, a) : cudaLaunchKernelEx(&cfg, rope_append_kernel<true, false>, a);
    else
        e = interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<false, true>, a) : cudaLaunchKernelEx(&cfg, rope_append_kernel<false, false>, a);
    return launched(e);
}
