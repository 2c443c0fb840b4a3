// kv_page_append_b8: the live rows of every sequence coded into its pages.
//
// A scale covers 16 positions of one head, so the unit of work is one such block of K or of V: its largest new
// magnitude gives the scale, and older rows of the block are coded again if the scale has grown.  One warp takes
// one block: half a warp holds a row (8 elements a lane), eight 16-byte loads a lane are in flight at once, the
// block's maximum is one integer warp reduction (magnitudes order like their bits), and nothing is read twice.
// Bytes: 2 read and 1 written per element.  A prompt of 16,384 rows of 8 heads (101 MB) takes 19.9 us, 5.1 TB/s; with
// a division wherever x (1 / s) came near a place where the code could change it took 35.8 us, because quotients of
// 8-bit significands are often such places.  A decode step's few rows are bound by the launch (4.6 us for 64 x 6).
#include "codec_dev.cuh"
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace va {
namespace paged {

constexpr int kAppendWarps = 4;

struct AppendArgs {
    const uint16_t *k_new, *v_new;
    const int32_t *n_live, *lens, *table;
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    int32_t* dev_status;
    int n_seqs, n_rows, n_kv, max_pages, n_pages, n_blocks;   // n_blocks: most blocks that one sequence's rows touch
};

// Eight quotients of magnitudes up to the largest code to eight codes.
template <bool kInt8>
__device__ __forceinline__ uint2 round8(const float (&q)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (kInt8) {
            // q + 1.5 x 2^23 is rounded to a whole number, ties to even; its lowest byte is the code
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fadd_rn(q[4 * h + i], 12582912.0f));
            w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        } else {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[4 * h + 1]), "f"(q[4 * h]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[4 * h + 3]), "f"(q[4 * h + 2]));
            w[h] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Eight floats to the codes of their correctly rounded quotients x / s.  inv is 1 / s correctly rounded, and
// q' = q + (x - q s) inv with q = x inv is then the correctly rounded quotient (P. Markstein, Computation of elementary
// functions on the IBM RISC System/6000 processor, 1990; his condition that q be within one unit in the last place does
// not always hold here, but the tests compare the codes with those of x / s for every significand of a bf16 x and of a
// block's largest value, and for every code coded again from one such scale to another).  `careful`: infinities
// among the x, or s so small that the remainder has no digits; these are divided and clamped.
template <bool kInt8>
__device__ __forceinline__ uint2 code8(const float (&x)[8], float s, float inv, bool careful) {
    float q[8];
    if (careful) {
        const float most = top_code(kInt8);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = s > 0.0f ? fminf(fmaxf(__fdiv_rn(x[i], s), -most), most) : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float near = __fmul_rn(x[i], inv);
            q[i] = __fmaf_rn(__fmaf_rn(-near, s, x[i]), inv, near);
        }
    }
    return round8<kInt8>(q);
}

template <bool kInt8>
__global__ void __launch_bounds__(32 * kAppendWarps, 8) append_kernel(const AppendArgs a) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, half = lane >> 4, li = lane & 15;
    const long long unit = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    // heads fastest: neighbouring warps read neighbouring rows of k_new / v_new
    const int h = (int)(unit % a.n_kv);
    long long rest = unit / a.n_kv;
    const bool is_v = rest & 1;
    rest >>= 1;
    const int i = (int)(rest % a.n_blocks);
    const long long b = rest / a.n_blocks;
    if (b >= a.n_seqs) return;
    const Seq sq = load_seq(a.lens, a.n_live, (int)b, a.n_rows, a.max_pages);
    const int start = sq.len - sq.live;
    const int block = start / kBlock + i;
    int status = sq.status;
    // (blocks are compared, not positions: a block behind the last may begin past 2^31)
    if (sq.live > 0 && block <= (sq.len - 1) / kBlock) {
        const int p0 = block * kBlock;
        // the rows on their way before the page is known
        const uint16_t* src = (is_v ? a.v_new : a.k_new) + ((size_t)b * a.n_rows * a.n_kv + h) * kD + 8 * li;
        uint4 raw[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int p = p0 + 2 * r + half;
            raw[r] = make_uint4(0u, 0u, 0u, 0u);
            if (p >= start && p < sq.len)
                raw[r] = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)(p - start) * a.n_kv * kD));
        }
        const int page = __ldcg(a.table + b * a.max_pages + block / kBlocks);
        if (page < 0 || page >= a.n_pages) {
            status |= VA_DEV_BAD_PAGE;
        } else {
            const int part = block % kBlocks;
            const size_t head = (size_t)page * a.n_kv + h;
            uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + head * kHeadBytes + part * kBlock * kD + 8 * li;
            float* scale = (is_v ? a.v_scale : a.k_scale) + head * kBlocks + part;
            const bool older = p0 < start;
            const float was = older ? __ldcg(scale) : 0.0f;
            // the block's largest magnitude, two elements at a time
            uint32_t top = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[r].x & 0x7FFF7FFFu, raw[r].y & 0x7FFF7FFFu),
                                             __vmaxu2(raw[r].z & 0x7FFF7FFFu, raw[r].w & 0x7FFF7FFFu)));
            top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xFFFFu));
            const bool special = top >= 0x7F80u;
            if (special) {
                // an infinity or NaN somewhere: the largest finite one instead, and NaN becomes 0
                status |= VA_DEV_NONFINITE;
                top = 0;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    uint32_t* w = reinterpret_cast<uint32_t*>(&raw[r]);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t m = (w[c] >> (16 * e)) & 0x7FFFu;
                            if (m > 0x7F80u) w[c] &= e ? 0x0000FFFFu : 0xFFFF0000u;
                            if (m < 0x7F80u) top = max(top, m);
                        }
                }
                top = __reduce_max_sync(0xffffffffu, top);
            }
            const float fresh = __fdiv_rn(__uint_as_float(top << 16), top_code(kInt8));
            const float s = older ? fmaxf(fresh, was) : fresh;
            // (the remainder is a multiple of 2^-56 s where a code depends on it)
            const bool careful = special || !(s > 8.3e-25f);
            const float inv = __frcp_rn(s);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int p = p0 + 2 * r + half;
                uint2* dst = reinterpret_cast<uint2*>(codes + (2 * r + half) * kD);
                if (p >= start && p < sq.len) {
                    float x[8];
                    const uint32_t w[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x[2 * c] = __uint_as_float(w[c] << 16);
                        x[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
                    }
                    *dst = code8<kInt8>(x, s, inv, careful);
                } else if (p < start && s > was) {
                    const uint2 c = *dst;
                    float lo[4], hi[4], x[8];
                    decode4<kInt8>(c.x, lo);
                    decode4<kInt8>(c.y, hi);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = __fmul_rn(lo[e], was);
                        x[4 + e] = __fmul_rn(hi[e], was);
                    }
                    *dst = code8<kInt8>(x, s, inv, careful);
                }
            }
            if (lane == 0) *scale = s;
        }
    }
    if (status && a.dev_status && lane == 0) atomicOr(a.dev_status, status);
}

}  // namespace paged
}  // namespace va

extern "C" va_status kv_page_append_b8(const va_bf16* k_new, const va_bf16* v_new, int n_seqs, int n_rows,
                                       int n_kv_heads, const int32_t* n_live, const int32_t* lens,
                                       const int32_t* table, int max_pages, void* k_codes, void* v_codes,
                                       float* k_scale, float* v_scale, int n_pages, int format, int32_t* dev_status,
                                       va_stream stream) {
    using namespace va::paged;
    if (!k_new || !v_new || !n_live || !lens || !table || !aligned16(k_new) || !aligned16(v_new)) return VA_INVALID_ARG;
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || n_rows < 1 || n_rows > (1 << 24)) return VA_INVALID_ARG;
    if (max_pages < 1 || max_pages > 0x7FFFFFFF / kPage) return VA_INVALID_ARG;
    if (format != VA_B8_E4M3 && format != VA_B8_INT8) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, 1, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    AppendArgs a;
    a.k_new = k_new; a.v_new = v_new;
    a.n_live = n_live; a.lens = lens; a.table = table;
    a.k_codes = static_cast<uint8_t*>(k_codes); a.v_codes = static_cast<uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.dev_status = dev_status;
    a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_kv = n_kv_heads; a.max_pages = max_pages; a.n_pages = n_pages;
    a.n_blocks = (n_rows + 2 * kBlock - 2) / kBlock;
    const long long units = (long long)n_seqs * a.n_blocks * n_kv_heads * 2;
    const long long ctas = (units + kAppendWarps - 1) / kAppendWarps;
    if (ctas > 0x7FFFFFFFll) return VA_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)ctas), dim3(32 * kAppendWarps), 0, (cudaStream_t)stream);
    return launched(format == VA_B8_INT8 ? cudaLaunchKernelEx(&cfg, append_kernel<true>, a)
                                         : cudaLaunchKernelEx(&cfg, append_kernel<false>, a));
}
