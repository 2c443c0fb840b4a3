// va_beam_select: beam search's selection over beams and vocabulary.
//
// One launch, three levels.  A CTA per (8,192-logit tile, row) reads its logits once: it forms the tile's maximum
// m and sum of exp(l - m) and collects the tile's k best keys as the sampler does, but forms keys only of the few
// logits at or above a bound (a 64-bit key of every logit took ten times the loads: 117 us for 32 x 8 x 151,669).  The last CTA of a row to
// arrive merges the tiles: log-sum-exp in 64 bits from the tiles' (m, sum), the row's k best keys, and their
// scores in 64 bits.  The last row of a request to arrive merges the hypotheses.  Every order is fixed by the
// keys, so the arrivals' order changes nothing.
// Bytes: the logits once; what a tile hands on (k keys) is 1/1000 of that.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "beam_select.h"
#include "paged.cuh"
#include "tc_ptx.cuh"
#include "topk_dev.cuh"
#include "va_internal.cuh"

namespace va {
namespace beam {

using namespace smp;

constexpr int kMaxRows = VA_BEAM_MAX_GROUPS * VA_BEAM_MAX_BEAMS;
constexpr size_t kCounterBytes = sizeof(unsigned) * ((size_t)kMaxRows + VA_BEAM_MAX_GROUPS);
constexpr int kMaxTiles = VA_SAMPLE_MAX_VOCAB / kTileLogits;          // 32
constexpr int kMaxMerge = kMaxK * kMaxTiles;                          // a row's tile keys
constexpr int kMaxFinal = kMaxK * VA_BEAM_MAX_BEAMS;                  // a request's candidates
constexpr int kWarps = kThreads / 32;

struct BeamSmem {
    uint64_t cand[kMaxMerge];   // tile: its candidates; row and request: the candidates that are ranked
    uint64_t red[kWarps];
    uint32_t wmin[kWarps];
    float fred[kWarps], fsum[kWarps];
    uint64_t all[kMaxMerge];    // row: every tile's keys; request: every hypothesis' score keys
    int32_t tok[kMaxFinal];     // request: their tokens
    int16_t who[kMaxFinal];     // request: which candidate a ranked key is
    uint64_t top[kMaxK];
    uint64_t tau;
    double max, log_sum;
    int n_cand, last;
};

struct BeamArgs {
    const void* logits;
    long long stride;
    const float* scores;
    const int32_t* finished;
    int32_t *parents, *tokens;
    float* out_scores;
    unsigned *row_count, *group_count;
    uint64_t* tile_keys;       // [rows][tiles][k]
    float2* tile_stats;        // [rows][tiles] (maximum, sum of exp(l - maximum))
    uint64_t* row_keys;        // [rows][k] order-preserving images of the scores, 0 = none
    int32_t* row_tokens;       // [rows][k]
    int vocab, n_beams, k, end_token;
};

// Order-preserving image of a score: 0 for -inf and NaN (no candidate).
__device__ __forceinline__ uint64_t score_key(double s) {
    if (!(s > -INFINITY)) return 0ull;
    if (s == 0.0) s = 0.0;
    const uint64_t b = (uint64_t)__double_as_longlong(s);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_score(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

// One arrival (release of the block's stores before it, acquire of the others'); every thread learns whether it
// was the last of n.  The last one resets the counter.
__device__ __forceinline__ bool arrive_last(unsigned* counter, int n, int* flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned prev;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(counter) : "memory");
        *flag = prev == (unsigned)(n - 1);
        if (*flag) *counter = 0u;
    }
    __syncthreads();
    return *flag != 0;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 3) beam_select_kernel(const BeamArgs a) {
    __shared__ BeamSmem sm;
    constexpr int kVec = kBf16 ? 8 : 4, kBytes = kBf16 ? 2 : 4;   // logits per 16 bytes
    const int tile = blockIdx.x, row = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_tiles = gridDim.x, k = a.k, first = tile * kTileLogits;
    const unsigned char* src = static_cast<const unsigned char*>(a.logits) + (size_t)row * a.stride * kBytes;
    ptx::griddep_launch_dependents();
    if (tid == 0) {   // pulled into L2 before the dependency resolves, as in the sampler
        const int n = min(kTileLogits, a.vocab - first) * kBytes & ~15;
        if (n > 0) ptx::bulk_prefetch_l2(src + (size_t)first * kBytes, (uint32_t)n);
    }
    ptx::griddep_wait();
    const bool done = a.finished && __ldcg(a.finished + row) != 0;
    if (done && tile > 0) return;
    const float base = __ldcg(a.scores + row);
    if (!done) {
        // ------------------------------------------------------------ tile
        float f[kPerThread];
        const int n_in = min(kTileLogits, a.vocab - first);
        uint4 raw[kPerThread / kVec];
#pragma unroll
        for (int i = 0; i < kPerThread / kVec; ++i) {
            const int at = (i * kThreads + tid) * kVec;
            if (at + kVec <= n_in) {
                raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)(first + at) * kBytes));
            } else {   // the row's end: entry by entry, -inf behind it
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (kBf16) {
                        uint32_t v = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int x = at + 2 * c + e;
                            v |= (x < n_in ? (uint32_t)*reinterpret_cast<const uint16_t*>(src + (size_t)(first + x) * 2) : 0xFF80u)
                                 << (16 * e);
                        }
                        w[c] = v;
                    } else {
                        const int x = at + c;
                        w[c] = x < n_in ? *reinterpret_cast<const uint32_t*>(src + (size_t)(first + x) * 4) : 0xFF800000u;
                    }
                }
                raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        float mine = -INFINITY;      // the thread's largest (NaN is passed over)
#pragma unroll
        for (int i = 0; i < kPerThread / kVec; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float x = kBf16 ? __uint_as_float((c & 1) ? (w[c / 2] & 0xFFFF0000u) : (w[c / 2] << 16))
                                      : __uint_as_float(w[c & 3]);
                f[i * kVec + c] = x;
                mine = fmaxf(mine, x);
            }
        }
        // The tile's maximum, and tau, a lower bound of its k-th largest logit: with f warps whose 32 threads all hold
        // logits and j = ceil(k / f), the smallest over those warps of the warp's j-th largest distinct thread maximum
        // (one warp-wide maximum a round).  Fewer than 32 threads of logits: every logit is a candidate.
        const int full_warps = min(kThreads, (n_in + kVec - 1) / kVec) / 32;
        const int rounds = full_warps > 0 ? (k + full_warps - 1) / full_warps : 1;
        uint32_t v = ord_bits(mine), low = 0u;
        for (int r = 0; r < rounds; ++r) {
            low = __reduce_max_sync(0xffffffffu, v);
            if (r == 0 && lane == 0) sm.fred[warp] = ord_to_float(low);
            v = v == low ? 0u : v;
        }
        if (lane == 0) sm.wmin[warp] = warp < full_warps ? low : 0xFFFFFFFFu;
        if (tid == 0) sm.n_cand = 0;
        __syncthreads();
        float mx = sm.fred[0];
        uint32_t tau_bits = sm.wmin[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            mx = fmaxf(mx, sm.fred[w]);
            tau_bits = min(tau_bits, sm.wmin[w]);
        }
        if (full_warps == 0) tau_bits = 0u;
        // candidates are at or above tau and above -inf (tau_bits 0 and NaN's image: all that are above -inf)
        const float tau = tau_bits > ord_bits(-INFINITY) ? ord_to_float(tau_bits) : -FLT_MAX;
        // exp(l - mx) as 2^(l log2 e + off): within 2^-22 for the terms that weigh anything, but for the rounding of
        // off, which all share and which is taken out of their sum.  (A maximum that is infinite or so large that
        // off would not hold its digits: the difference first.)
        const float l2e = 1.4426950408889634f;
        const bool plain = fabsf(mx) < 1024.0f;
        const float off = plain ? -mx * l2e : 0.0f, shared_error = plain ? fmaf(mx, l2e, off) : 0.0f;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        unsigned bits = 0;
        if (plain) {
#pragma unroll
            for (int e = 0; e < kPerThread; ++e)
                if (f[e] == f[e]) sum[e & 3] += ptx::ex2(fmaf(f[e], l2e, off));
        } else if (mx > -INFINITY) {
#pragma unroll
            for (int e = 0; e < kPerThread; ++e)
                if (f[e] == f[e]) sum[e & 3] += f[e] == mx ? 1.0f : ptx::ex2((f[e] - mx) * l2e);
        }
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) bits |= f[e] >= tau ? 1u << e : 0u;
        float part = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == 0) sm.fsum[warp] = part;
        // compaction: a warp's candidates take consecutive places; their values are read again (few are)
        const int cnt = __popc(bits);
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        int slot = 0;
        if (lane == 31 && incl > 0) slot = atomicAdd(&sm.n_cand, incl);
        slot = __shfl_sync(0xffffffffu, slot, 31) + incl - cnt;
        for (unsigned rest = bits; rest != 0; rest &= rest - 1) {
            const int e = __ffs(rest) - 1;
            const int at = first + ((e / kVec) * kThreads + tid) * kVec + e % kVec;
            const float x = kBf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(src)[at] << 16)
                                  : reinterpret_cast<const float*>(src)[at];
            if (slot < kMaxCand) sm.cand[slot] = make_key(x, at);
            ++slot;
        }
        __syncthreads();
        const int n_cand = sm.n_cand;
        if (tid == 0) {
            float all = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) all += sm.fsum[w];
            a.tile_stats[(size_t)row * n_tiles + tile] = make_float2(mx, mx > -INFINITY ? fmaf(all, -0.69314718f * shared_error, all) : 0.0f);
        }
        uint64_t* keys_out = a.tile_keys + ((size_t)row * n_tiles + tile) * k;
        if (n_cand <= kMaxCand) {
            // rank by counting: a candidate goes to the place of the number of larger ones, if that is below k
            for (int c = tid; c < n_cand; c += kThreads) {
                const uint64_t kc = sm.cand[c];
                int rank = 0;
#pragma unroll 8
                for (int o = 0; o < n_cand; ++o) rank += sm.cand[o] > kc;
                if (rank < k) keys_out[rank] = kc;
            }
            for (int r = n_cand + tid; r < k; r += kThreads) keys_out[r] = 0ull;
        } else {
            // many equal logits at the bound: k rounds of block-wide maximum over every logit
            uint64_t taken = ~0ull;
            for (int r = 0; r < k; ++r) {
                uint64_t best = 0;
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) {
                    const uint64_t kv = f[e] > -INFINITY ? make_key(f[e], first + ((e / kVec) * kThreads + tid) * kVec + e % kVec) : 0ull;
                    best = kv < taken && kv > best ? kv : best;
                }
                best = block_max_u64(best, sm.red);
                if (tid == 0) keys_out[r] = best;
                taken = best;
            }
        }
        if (!arrive_last(a.row_count + row, n_tiles, &sm.last)) return;
        // -------------------------------------------------------- row
        const uint64_t* rw = a.tile_keys + (size_t)row * n_tiles * k;
        const int total = n_tiles * k;
        for (int e = tid; e < total; e += kThreads) sm.all[e] = __ldcg(rw + e);
        __syncthreads();
        if (warp == 0) {
            // a lower bound of the row's k-th key: the smallest of every tile's ceil(k / tiles)-th
            const int m = min(k, (k + n_tiles - 1) / n_tiles);
            uint64_t b = ~0ull;
            if (lane < n_tiles) b = sm.all[lane * k + m - 1];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t w = __shfl_xor_sync(0xffffffffu, b, o);
                b = w < b ? w : b;
            }
            if (lane == 0) {
                sm.tau = b;
                sm.n_cand = 0;
            }
            // log-sum-exp over the tiles, one a lane
            const float2 st = lane < n_tiles ? __ldcg(a.tile_stats + (size_t)row * n_tiles + lane) : make_float2(-INFINITY, 0.0f);
            float top = st.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            double s = st.x == -INFINITY ? 0.0 : (st.x == top ? (double)st.y : (double)(st.y * expf(st.x - top)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) {
                sm.max = (double)top;
                sm.log_sum = log(s);
            }
        } else if (warp == 1) {
            sm.top[lane] = 0ull;
        }
        __syncthreads();
        const uint64_t lb = sm.tau;
        for (int e = tid; e < total; e += kThreads) {
            const uint64_t kv = sm.all[e];
            if (kv >= lb && kv != 0ull) sm.cand[atomicAdd(&sm.n_cand, 1)] = kv;
        }
        __syncthreads();
        const int nc = sm.n_cand;
        for (int c = tid; c < nc; c += kThreads) {
            const uint64_t kc = sm.cand[c];
            int rank = 0;
#pragma unroll 8
            for (int o = 0; o < nc; ++o) rank += sm.cand[o] > kc;
            if (rank < k) sm.top[rank] = kc;
        }
        __syncthreads();
        if (tid < k) {
            const uint64_t kv = sm.top[tid];
            uint64_t sk = 0ull;
            if (kv != 0ull) {
                const double l = (double)ord_to_float((uint32_t)(kv >> 32));
                const double above = l == sm.max ? 0.0 : l - sm.max;
                sk = score_key((double)base + (above - sm.log_sum));
            }
            a.row_keys[(size_t)row * k + tid] = sk;
            a.row_tokens[(size_t)row * k + tid] = key_index(kv);
        }
    } else if (tid < k) {
        a.row_keys[(size_t)row * k + tid] = tid == 0 ? score_key((double)base) : 0ull;
        a.row_tokens[(size_t)row * k + tid] = a.end_token;
    }
    // ---------------------------------------------------------------- request
    const int group = row / a.n_beams;
    if (!arrive_last(a.group_count + group, a.n_beams, &sm.last)) return;
    const int total = a.n_beams * k;
    const size_t at = (size_t)group * total;
    for (int e = tid; e < total; e += kThreads) {
        sm.all[e] = __ldcg(a.row_keys + at + e);
        sm.tok[e] = __ldcg(a.row_tokens + at + e);
    }
    __syncthreads();
    if (warp == 0) {   // a lower bound of the k-th score: the smallest of every hypothesis' ceil(k / beams)-th
        const int m = (k + a.n_beams - 1) / a.n_beams;
        uint64_t b = lane < a.n_beams ? sm.all[lane * k + m - 1] : ~0ull;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t w = __shfl_xor_sync(0xffffffffu, b, o);
            b = w < b ? w : b;
        }
        if (lane == 0) {
            sm.tau = b;
            sm.n_cand = 0;
        }
    }
    __syncthreads();
    const uint64_t lb = sm.tau;
    for (int e = tid; e < total; e += kThreads) {
        const uint64_t kv = sm.all[e];
        if (kv >= lb && kv != 0ull) {
            const int i = atomicAdd(&sm.n_cand, 1);
            sm.cand[i] = kv;
            sm.who[i] = (int16_t)e;
        }
    }
    __syncthreads();
    const int nc = sm.n_cand;
    const size_t out = (size_t)group * k;
    for (int c = tid; c < nc; c += kThreads) {
        const uint64_t kc = sm.cand[c];
        const int e = sm.who[c];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < nc; ++o) rank += sm.cand[o] > kc || (sm.cand[o] == kc && sm.who[o] < e);
        if (rank < k) {
            a.parents[out + rank] = e / k;
            a.tokens[out + rank] = sm.tok[e];
            a.out_scores[out + rank] = (float)key_score(kc);
        }
    }
    for (int r = nc + tid; r < k; r += kThreads) {
        a.parents[out + r] = -1;
        a.tokens[out + r] = -1;
        a.out_scores[out + r] = -INFINITY;
    }
}

}  // namespace beam
}  // namespace va

namespace {
int beam_tiles(int vocab) { return (vocab + VA_SAMPLE_TILE - 1) / VA_SAMPLE_TILE; }
}  // namespace

extern "C" {

size_t va_beam_workspace_bytes(int n_groups, int n_beams, int vocab, int n_out) {
    if (n_groups < 1 || n_groups > VA_BEAM_MAX_GROUPS || n_beams < 1 || n_beams > VA_BEAM_MAX_BEAMS || vocab < 1 ||
        vocab > VA_SAMPLE_MAX_VOCAB || n_out < 1 || n_out > VA_SAMPLE_MAX_K)
        return 0;
    // the counters first, at places that do not depend on the shape; then per row the tiles' keys and
    // statistics, and the row's scores and tokens
    const size_t rows = (size_t)n_groups * n_beams, tiles = beam_tiles(vocab);
    return va::beam::kCounterBytes + rows * tiles * (8 * (size_t)n_out + 8) + rows * n_out * 12;
}

va_status va_beam_select(const void* logits, int format, int64_t row_stride, int n_groups, int n_beams, int vocab,
                         const float* scores, const int32_t* finished, int end_token, int n_out, int32_t* parents,
                         int32_t* tokens, float* out_scores, void* workspace, size_t workspace_bytes,
                         va_stream stream) {
    const size_t need = va_beam_workspace_bytes(n_groups, n_beams, vocab, n_out);
    if (need == 0 || !logits || !scores || !parents || !tokens || !out_scores || !workspace) return VA_INVALID_ARG;
    if (format != VA_LOGITS_F32 && format != VA_LOGITS_BF16) return VA_INVALID_ARG;
    if (!va::paged::aligned16(logits) || !va::paged::aligned16(workspace) || workspace_bytes < need) return VA_INVALID_ARG;
    if (row_stride < vocab || row_stride % (format == VA_LOGITS_BF16 ? 8 : 4) != 0) return VA_INVALID_ARG;
    if (finished && (end_token < 0 || end_token >= vocab)) return VA_INVALID_ARG;
    const size_t rows = (size_t)n_groups * n_beams;
    const int tiles = beam_tiles(vocab);
    va::beam::BeamArgs a;
    a.logits = logits; a.stride = row_stride; a.scores = scores; a.finished = finished;
    a.parents = parents; a.tokens = tokens; a.out_scores = out_scores;
    unsigned char* p = static_cast<unsigned char*>(workspace);
    a.row_count = reinterpret_cast<unsigned*>(p);
    a.group_count = a.row_count + va::beam::kMaxRows;
    p += va::beam::kCounterBytes;
    a.tile_keys = reinterpret_cast<uint64_t*>(p);
    p += rows * tiles * n_out * 8;
    a.tile_stats = reinterpret_cast<float2*>(p);
    p += rows * tiles * 8;
    a.row_keys = reinterpret_cast<uint64_t*>(p);
    p += rows * n_out * 8;
    a.row_tokens = reinterpret_cast<int32_t*>(p);
    a.vocab = vocab; a.n_beams = n_beams; a.k = n_out; a.end_token = end_token;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3(tiles, (unsigned)rows), dim3(va::smp::kThreads), 0, (cudaStream_t)stream);
    return va::paged::launched(format == VA_LOGITS_BF16
                                   ? cudaLaunchKernelEx(&cfg, va::beam::beam_select_kernel<true>, a)
                                   : cudaLaunchKernelEx(&cfg, va::beam::beam_select_kernel<false>, a));
}

}  // extern "C"
