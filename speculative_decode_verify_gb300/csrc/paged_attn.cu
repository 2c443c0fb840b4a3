// verify_attn_paged_b8: the call, and the second of its two launches, which merges what the split kernels
// (paged_attn.cuh, paged_attn_tc.cuh) left in parts and writes the rows that see nothing.
#include <cmath>

#include "paged_plan.cuh"

namespace va {
namespace tc {
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();   // attn_tc.cu
}  // namespace tc

namespace paged {

cudaError_t launch_attn_e4m3(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream);
cudaError_t launch_attn_int8(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream);

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMost = kMaxCtas / kJoinWarps;   // most parts of a warp

// CTA (unit, y): unit = (sequence, KV head); its (row, query head) pairs y, y + gridDim.y, ..
// Few parts: a warp a pair.  Many (a long history over many CTAs): the warps share a pair's parts, each a
// consecutive run, and join through shared memory; the order is fixed.
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnPagedArgs a) {
    __shared__ long long sums[3 * kJoinWarps];
    __shared__ float4 acc_s[kJoinWarps][32];
    __shared__ float2 ml_s[kJoinWarps];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.n_kv, h = blockIdx.x % a.n_kv, heads = a.n_kv * a.group;
    // costs before this sequence, and of all; tiles of all (the deal of the split kernel)
    long long before = 0, total = 0, tiles = 0;
    for (int s = tid; s < a.n_seqs; s += kJoinThreads) {
        const Seq q = load_seq(a.lens, a.n_live, s, a.n_rows, a.max_pages);
        const int n = span_of(q.len, q.live, a.window).n;
        const long long cost = n > 0 ? (long long)(n + kSegCost) * a.n_kv : 0;
        total += cost;
        tiles += (long long)n * a.n_kv;
        if (s < b) before += cost;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
        tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    }
    if (lane == 0) {
        sums[warp] = before;
        sums[kJoinWarps + warp] = total;
        sums[2 * kJoinWarps + warp] = tiles;
    }
    __syncthreads();
    before = total = tiles = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        before += sums[w];
        total += sums[kJoinWarps + w];
        tiles += sums[2 * kJoinWarps + w];
    }
    const Seq sq = load_seq(a.lens, a.n_live, b, a.n_rows, a.max_pages);
    const int n_tiles = span_of(sq.len, sq.live, a.window).n;
    // padding rows
    for (int c = blockIdx.y * kJoinWarps + warp; c < (a.n_rows - sq.live) * a.group; c += gridDim.y * kJoinWarps) {
        const size_t row = ((size_t)b * a.n_rows + sq.live + c / a.group) * heads + h * a.group + c % a.group;
        reinterpret_cast<uint2*>(a.out + row * kD)[lane] = make_uint2(0u, 0u);
        if (lane == 0 && a.out_lse) a.out_lse[row] = -INFINITY;
    }
    if (n_tiles == 0) return;
    const int n_ctas = (int)min((long long)a.n_ctas, tiles);
    const long long first = before + (long long)h * (n_tiles + kSegCost);    // this head's first cost
    auto cta_of = [&](long long y) {
        return total < (1ll << 24) ? (int)(((unsigned)(y + 1) * (unsigned)n_ctas - 1u) / (unsigned)total)
                                   : (int)(((y + 1) * n_ctas - 1) / total);
    };
    const int c_first = cta_of(first + kSegCost), c_last = cta_of(first + kSegCost + n_tiles - 1);
    if (c_first == c_last) return;   // the split kernel has written the rows
    const int parts = c_last - c_first + 1;
    // the part of a CTA is its first segment's, but for the head's first CTA if the head begins inside it
    const size_t first_place = (size_t)(2 * c_first + (cta_begin(c_first, n_ctas, total) >= first ? 0 : 1)) * kMaxCols;
    auto place = [&](int p) { return p == 0 ? first_place : (size_t)(2 * (c_first + p)) * kMaxCols; };
    const bool shared = parts > kMost;
    const int n_cols = sq.live * a.group, step = shared ? (int)gridDim.y : (int)gridDim.y * kJoinWarps;
    for (int col = shared ? (int)blockIdx.y : (int)blockIdx.y * kJoinWarps + warp; col < n_cols; col += step) {
        const int p0 = shared ? parts * warp / kJoinWarps : 0, p1 = shared ? parts * (warp + 1) / kJoinWarps : parts;
        // all of the warp's parts in flight at once: their sums, and (one a lane) their references
        float4 v[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (p0 + i < p1) v[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (place(p0 + i) + col) * kD) + lane);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < p1 - p0) ml = __ldcg(a.part_ml + place(p0 + lane) + col);
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float by = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.0f) : exp2f(ml.x - top);
        float sum = by * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (p0 + i < p1) {
                const float w = __shfl_sync(0xffffffffu, by, i);
                acc.x += w * v[i].x;
                acc.y += w * v[i].y;
                acc.z += w * v[i].z;
                acc.w += w * v[i].w;
            }
        if (shared) {
            __syncthreads();
            acc_s[warp][lane] = acc;
            if (lane == 0) ml_s[warp] = make_float2(top, sum);
            __syncthreads();
            if (warp != 0) continue;
            top = ml_s[0].x;
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, ml_s[w].x);
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float2 one = ml_s[w];
                const float f = one.x == -INFINITY ? (one.y != one.y ? one.y : 0.0f) : exp2f(one.x - top);
                const float4 v = acc_s[w][lane];
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
                sum += f * one.y;
            }
        }
        const int head = h * a.group + col % a.group;
        const size_t row = ((size_t)b * a.n_rows + col / a.group) * heads + head;
        const Finish f = finish(top, sum, a.sink, head);
        store_row(a.out + row * kD + 4 * lane, make_float4(acc.x * f.by, acc.y * f.by, acc.z * f.by, acc.w * f.by));
        if (lane == 0 && a.out_lse) a.out_lse[row] = f.lse;
    }
}

// A pool as rows of 128 codes; boxes of one head's 64 positions, swizzled.
static bool encode_pool(CUtensorMap* map, const void* base, int rows) {
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)kD};
    const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)kPage};
    const cuuint32_t elem[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace paged
}  // namespace va

extern "C" {

size_t va_paged_workspace_bytes(int n_seqs, int n_rows, int n_kv_heads, int group) {
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || n_rows < 1 || n_rows > VA_MAX_ROWS || n_kv_heads < 1 ||
        n_kv_heads > VA_PAGED_MAX_KV_HEADS || group < 1 || group > VA_PAGED_MAX_GROUP)
        return 0;
    return va::paged::kWorkspaceBytes;   // two parts a CTA, whatever the batch
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
    const int sms = va::device_sm_count();
    AttnPagedArgs a;
    a.q = q; a.n_live = n_live; a.lens = lens; a.table = table;
    a.k_codes = static_cast<const uint8_t*>(k_codes); a.v_codes = static_cast<const uint8_t*>(v_codes);
    a.k_scale = k_scale; a.v_scale = v_scale; a.sink = sink; a.out = out; a.out_lse = out_lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + kPartFloats);
    a.dev_status = dev_status;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_kv = n_kv_heads; a.group = group;
    a.max_pages = max_pages; a.n_pages = n_pages; a.window = window;
    a.n_ctas = sms > 0 && sms < kMaxCtas ? sms : kMaxCtas;
    CUtensorMap mk, mv;      // (paged_attn_tc.cuh takes none)
    const int pool_rows = n_pages * n_kv_heads * kPage;      // below 2^31 (check_pool)
    if (n_rows * group <= kFewPairs && !(encode_pool(&mk, k_codes, pool_rows) && encode_pool(&mv, v_codes, pool_rows)))
        return VA_CUDA_ERROR;
    st = launched((format == VA_B8_INT8 ? launch_attn_int8 : launch_attn_e4m3)(
        a, mk, mv, (cudaStream_t)stream));
    if (st != VA_OK) return st;
    // about one CTA an SM: a unit each where there are enough, else its pairs are shared out
    const int units = n_seqs * n_kv_heads, pairs = n_rows * group;
    const int share = units >= a.n_ctas ? 1 : (a.n_ctas + units - 1) / units;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)units, (unsigned)(share < pairs ? share : pairs)), dim3(kJoinThreads), 0,
                   (cudaStream_t)stream);
    return launched(cudaLaunchKernelEx(&cfg, attn_join_kernel, a));
}

}  // extern "C"
