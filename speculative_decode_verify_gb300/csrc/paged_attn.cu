// verify_attn_paged_b8: verify attention of a batch of sequences over their pages.
#include <cmath>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace va {
namespace paged {

struct AttnPagedArgs {
    const uint16_t* q;
    const int32_t *n_live, *lens, *table;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const float* sink;
    uint16_t* out;
    float* out_lse;
    int32_t* dev_status;
    float scale;
    int n_seqs, n_rows, n_kv, group, max_pages, n_pages, window;
};

// One warp per (sequence, row, query head): 32 keys at a time, a key a lane for the scores, four dimensions a
// lane for the output.
template <bool kInt8>
__global__ void __launch_bounds__(32) attn_paged_kernel(const AttnPagedArgs a) {
    __shared__ float qs[kD];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x, heads = a.n_kv * a.group;
    const int head = blockIdx.x % heads, r = blockIdx.x / heads % a.n_rows, b = blockIdx.x / heads / a.n_rows;
    const int h = head / a.group;
    const Seq sq = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
    int status = sq.status;
    const size_t row = ((size_t)b * a.n_rows + r) * heads + head;
    float m = -INFINITY, l = 0.0f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const bool live = r < sq.live;
    if (live) {
        for (int e = 0; e < 4; ++e) qs[lane + 32 * e] = __uint_as_float((uint32_t)a.q[row * kD + lane + 32 * e] << 16);
        __syncwarp();
        const int p = sq.len - sq.live + r;
        const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
        for (int j0 = lo / 32 * 32; j0 <= p; j0 += 32) {
            const int j = j0 + lane;
            const int page = __ldcg(a.table + (size_t)b * a.max_pages + j0 / kPage);
            if (page < 0 || page >= a.n_pages) {
                status |= VA_DEV_BAD_PAGE;
                continue;
            }
            const size_t base = (size_t)page * a.n_kv + h;
            float s = -INFINITY;
            if (j >= lo && j <= p) {
                const uint32_t* kr = reinterpret_cast<const uint32_t*>(a.k_codes + (base * kPage + j % kPage) * kD);
                float acc = 0.0f;
                for (int w = 0; w < kD / 4; ++w) {
                    float x[4];
                    decode4<kInt8>(__ldcg(kr + w), x);
                    for (int e = 0; e < 4; ++e) acc = fmaf(x[e], qs[4 * w + e], acc);
                }
                s = acc * __ldcg(a.k_scale + base * kBlocks + j % kPage / kBlock) * a.scale;
            }
            float mx = s;
            for (int o2 = 16; o2 > 0; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
            const float mn = fmaxf(m, mx);
            const float f = m == -INFINITY ? 0.0f : expf(m - mn);
            const float pr = s == -INFINITY ? 0.0f : expf(s - mn);
            m = mn;
            l = l * f + pr;
            for (int e = 0; e < 4; ++e) o[e] *= f;
            for (int t = 0; t < 32; ++t) {
                const float pt = __shfl_sync(0xffffffffu, pr, t);
                const int jt = j0 + t;
                if (jt < lo || jt > p) continue;
                float x[4];
                decode4<kInt8>(__ldcg(reinterpret_cast<const uint32_t*>(a.v_codes + (base * kPage + jt % kPage) * kD) + lane), x);
                const float vs = __ldcg(a.v_scale + base * kBlocks + jt % kPage / kBlock);
                for (int e = 0; e < 4; ++e) o[e] = fmaf(pt * vs, x[e], o[e]);
            }
        }
        for (int o2 = 16; o2 > 0; o2 >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
    }
    float L = -INFINITY;
    if (live) {
        const float sink = a.sink ? a.sink[head] : -INFINITY;
        const float top = fmaxf(m, sink);
        if (top != -INFINITY) {
            const float em = m == -INFINITY ? 0.0f : expf(m - top);
            const float total = l * em + (sink == -INFINITY ? 0.0f : expf(sink - top));
            for (int e = 0; e < 4; ++e) o[e] = total > 0.0f ? o[e] * em / total : 0.0f;
            L = top + logf(total);
        }
    }
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = __float_as_uint(o[e]);
        a.out[row * kD + 4 * lane + e] = (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    }
    if (lane == 0 && a.out_lse) a.out_lse[row] = L;
    if (lane == 0 && status && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace paged
}  // namespace va

extern "C" {

size_t va_paged_workspace_bytes(int n_seqs, int n_rows, int n_kv_heads, int group) {
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || n_rows < 1 || n_rows > VA_MAX_ROWS || n_kv_heads < 1 ||
        n_kv_heads > VA_PAGED_MAX_KV_HEADS || group < 1 || group > VA_PAGED_MAX_GROUP)
        return 0;
    return 256;
}

va_status verify_attn_paged_b8(const va_bf16* q, int n_seqs, int n_rows, int n_kv_heads, int group,
                               const int32_t* n_live, const int32_t* lens, const int32_t* table, int max_pages,
                               const void* k_codes, const void* v_codes, const float* k_scale, const float* v_scale,
                               int n_pages, int format, int window, float scale, const float* sink, void* workspace,
                               size_t workspace_bytes, va_bf16* out, float* out_lse, int32_t* dev_status,
                               va_stream stream) {
    using namespace va::paged;
    const size_t need = va_paged_workspace_bytes(n_seqs, n_rows, n_kv_heads, group);
    if (need == 0 || !q || !n_live || !lens || !table || !workspace || !out) return VA_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || workspace_bytes < need) return VA_INVALID_ARG;
    if (max_pages < 1 || max_pages > 0x7FFFFFFF / kPage || window < 0 || !std::isfinite(scale)) return VA_INVALID_ARG;
    if (format != VA_B8_E4M3 && format != VA_B8_INT8) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, 1, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    AttnPagedArgs a;
    a.q = q; a.n_live = n_live; a.lens = lens; a.table = table;
    a.k_codes = static_cast<const uint8_t*>(k_codes); a.v_codes = static_cast<const uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale; a.sink = sink; a.out = out; a.out_lse = out_lse;
    a.dev_status = dev_status; a.scale = scale;
    a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_kv = n_kv_heads; a.group = group;
    a.max_pages = max_pages; a.n_pages = n_pages; a.window = window;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)(n_seqs * n_rows * n_kv_heads * group)), dim3(32), 0, (cudaStream_t)stream);
    return launched(format == VA_B8_INT8 ? cudaLaunchKernelEx(&cfg, attn_paged_kernel<true>, a)
                                         : cudaLaunchKernelEx(&cfg, attn_paged_kernel<false>, a));
}

}  // extern "C"
