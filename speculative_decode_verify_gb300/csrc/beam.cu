// va_beam_select: beam search's selection over beams and vocabulary.
//
// One launch, three levels.  The (row, 8,192-logit tile) units are dealt evenly to four CTAs an SM; a run is a CTA's
// consecutive tiles of one row.  A CTA reads a tile's logits once (the next tile's are on their way into L2):
//   sums        every thread keeps its own maximum m and sum of exp(l - m) over the run
//   candidates  the run's k best keys so far are kept sorted in shared memory.  The first tile collects against a lower
//               bound of its k-th logit, as the sampler does; a later one only the logits above the k-th so far (its
//               indices are higher, so equal ones lose), few of which are left to rank.
// The last run of a row to arrive merges the runs: log-sum-exp in 64 bits, the row's k best keys and their scores in
// 64 bits.  The last row of a request merges the hypotheses.  Every order is fixed by the keys and by the deal, so the
// arrivals' order changes nothing.
// Bytes: the logits once; what a run hands on (k keys) is a thousandth of that.  A 64-bit key for every logit took
// 117 us for 32 x 8 x 151,669 bf16 logits, keys and a ranking for every tile's candidates 56 us; this takes 50 us with
// four CTAs an SM (52 with three, 59 with two), and with a list for every warp instead of the CTA's, which needs no
// barriers but eight times the insertions, 67 us.
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
    uint64_t cand[kMaxMerge];   // run: its best so far, then a tile's candidates; row and request: what is ranked
    uint64_t best[kMaxK];       // run: the new best
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
    uint64_t* run_keys;        // [rows][tiles][k]: the rows' runs in order (at most as many as tiles)
    float2* run_stats;         // [rows][tiles] (maximum, sum of exp(l - maximum))
    uint64_t* row_keys;        // [rows][k] order-preserving images of the scores, 0 = none
    int32_t* row_tokens;       // [rows][k]
    int vocab, n_beams, k, end_token, n_tiles, n_rows;
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

// `mine` arrivals of n (release of the block's stores before them, acquire of the others'); every thread learns
// whether they were the last.  The last one resets the counter.
__device__ __forceinline__ bool arrive_last(unsigned* counter, int mine, int n, int* flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned prev;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(prev) : "l"(counter), "r"(mine) : "memory");
        *flag = prev + (unsigned)mine == (unsigned)n;
        if (*flag) *counter = 0u;
    }
    __syncthreads();
    return *flag != 0;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamArgs a) {
    __shared__ BeamSmem sm;
    constexpr int kVec = kBf16 ? 8 : 4, kBytes = kBf16 ? 2 : 4;   // logits per 16 bytes
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_tiles = a.n_tiles, k = a.k;
    // this CTA's share of the (row, tile) units, in order
    const unsigned units = (unsigned)a.n_rows * n_tiles;      // at most 2^20, by fewer than 2^11 CTAs
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    auto row_at = [&](int row) { return static_cast<const unsigned char*>(a.logits) + (size_t)row * a.stride * kBytes; };
    auto prefetch = [&](int u) {
        if (tid == 0 && u < u1) {
            const int first = u % n_tiles * kTileLogits, n = min(kTileLogits, a.vocab - first) * kBytes & ~15;
            if (n > 0) ptx::bulk_prefetch_l2(row_at(u / n_tiles) + (size_t)first * kBytes, (uint32_t)n);
        }
    };
    ptx::griddep_launch_dependents();
    prefetch(u0);          // pulled into L2 before the dependency resolves, as in the sampler
    ptx::griddep_wait();
    const float l2e = 1.4426950408889634f;
    int run = 0;                            // tiles of the run so far
    float m = -INFINITY, sum = 0.0f;        // this thread's maximum of them, and its sum of exp(l - m)
    for (int u = u0; u < u1; ++u) {
        const int row = u / n_tiles, tile = u % n_tiles, first = tile * kTileLogits;
        const unsigned char* src = row_at(row);
        prefetch(u + 1);
        const bool done = a.finished && __ldcg(a.finished + row) != 0;
        const float base = __ldcg(a.scores + row);
        if (!done) {
            // -------------------------------------------------------- tile
            float f[kPerThread];
            const int n_in = min(kTileLogits, a.vocab - first);
#pragma unroll
            for (int i = 0; i < kPerThread / kVec; ++i) {
                const int at = (i * kThreads + tid) * kVec;
                uint32_t w[4];
                if (at + kVec <= n_in) {
                    const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)(first + at) * kBytes));
                    w[0] = raw.x;
                    w[1] = raw.y;
                    w[2] = raw.z;
                    w[3] = raw.w;
                } else {   // the row's end: entry by entry, -inf behind it
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
                }
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    const float x = kBf16 ? __uint_as_float((c & 1) ? (w[c / 2] & 0xFFFF0000u) : (w[c / 2] << 16))
                                          : __uint_as_float(w[c & 3]);
                    f[i * kVec + c] = fmaxf(x, -INFINITY);      // a NaN is no candidate: -inf
                }
            }
            float mine = -INFINITY;      // the thread's largest
#pragma unroll
            for (int e = 0; e < kPerThread; ++e) mine = fmaxf(mine, f[e]);
            // sums, as 2^(l log2 e + off); a maximum for which off has no digits takes the careful way
            if (mine > -INFINITY) {
                const float up = fmaxf(m, mine), off = -up * l2e;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) part[e & 3] += ptx::ex2(fmaf(f[e], l2e, off));
                float add = (part[0] + part[1]) + (part[2] + part[3]);
                if (!(fabsf(up) < 1024.0f)) {
                    add = 0.0f;
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) add += f[e] == up ? 1.0f : ptx::ex2((f[e] - up) * l2e);
                }
                sum = (m == up ? sum : (m == -INFINITY ? 0.0f : sum * ptx::ex2((m - up) * l2e))) + add;
                m = up;
            }
            // the bound that candidates have to pass
            const int held = run > 0 ? k : 0;
            float tau;
            if (run > 0) {
                const uint64_t kth = sm.cand[k - 1];
                tau = kth != 0ull ? ord_to_float((uint32_t)(kth >> 32) + 1u) : -FLT_MAX;   // the next larger float
            } else {
                // A lower bound of the tile's k-th largest logit: with f warps whose 32 threads all hold logits and
                // j = ceil(k / f), the smallest over those warps of the warp's j-th largest distinct thread maximum
                // (one warp-wide maximum a round).  Fewer than 32 threads of logits: every logit is a candidate.
                const int full_warps = min(kThreads, (n_in + kVec - 1) / kVec) / 32;
                const int rounds = full_warps > 0 ? (k + full_warps - 1) / full_warps : 1;
                uint32_t v = ord_bits(mine), low = 0u;
                for (int r = 0; r < rounds; ++r) {
                    low = __reduce_max_sync(0xffffffffu, v);
                    v = v == low ? 0u : v;
                }
                if (lane == 0) sm.wmin[warp] = warp < full_warps ? low : 0xFFFFFFFFu;
                __syncthreads();
                uint32_t least = sm.wmin[0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) least = min(least, sm.wmin[w]);
                if (full_warps == 0) least = 0u;
                tau = least > ord_bits(-INFINITY) ? ord_to_float(least) : -FLT_MAX;
            }
            unsigned bits = 0;
            if (mine >= tau) {
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) bits |= f[e] >= tau ? 1u << e : 0u;
            }
            if (tid == 0) sm.n_cand = held;
            if (__syncthreads_or(bits != 0)) {
                // compaction behind the best so far: a warp's candidates take consecutive places; the values are read
                // again (few are)
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
                    if (slot < held + kMaxCand) sm.cand[slot] = make_key(x, at);
                    ++slot;
                }
                if (tid < k) sm.best[tid] = 0ull;
                __syncthreads();
                int n = sm.n_cand;
                if (n > held + kMaxCand) {
                    // many equal logits at the bound: the tile's k best by k rounds of block-wide maximum
                    uint64_t taken = ~0ull;
                    for (int r = 0; r < k; ++r) {
                        uint64_t best = 0;
#pragma unroll
                        for (int e = 0; e < kPerThread; ++e) {
                            const uint64_t kv = f[e] >= tau ? make_key(f[e], first + ((e / kVec) * kThreads + tid) * kVec + e % kVec) : 0ull;
                            best = kv < taken && kv > best ? kv : best;
                        }
                        best = block_max_u64(best, sm.red);
                        if (tid == 0) sm.cand[held + r] = best;
                        taken = best;
                    }
                    n = held + k;
                    __syncthreads();
                }
                // rank by counting: a key goes to the place of the number of larger ones, if that is below k
                for (int c = tid; c < n; c += kThreads) {
                    const uint64_t kc = sm.cand[c];
                    int rank = 0;
#pragma unroll 8
                    for (int o = 0; o < n; ++o) rank += sm.cand[o] > kc;
                    if (rank < k && kc != 0ull) sm.best[rank] = kc;
                }
                __syncthreads();
                if (tid < k) sm.cand[tid] = sm.best[tid];
            } else if (run == 0 && tid < k) {
                sm.cand[tid] = 0ull;
            }
            __syncthreads();
            ++run;
            if (tile != n_tiles - 1 && u + 1 != u1) continue;
            // -------------------------------------------------------- the run's end
            const int c_first = (int)(((unsigned)(row * n_tiles + 1) * gridDim.x - 1u) / units);
            const int c_last = (int)(((unsigned)((row + 1) * n_tiles) * gridDim.x - 1u) / units);
            const int n_runs = c_last - c_first + 1;
            float top = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) sm.fred[warp] = top;
            __syncthreads();
            top = sm.fred[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.fred[w]);
            float all = m == top ? (top > -INFINITY ? sum : 0.0f) : (m == -INFINITY ? 0.0f : sum * ptx::ex2((m - top) * l2e));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            if (lane == 0) sm.fsum[warp] = all;
            __syncthreads();
            const size_t place = (size_t)row * n_tiles + (blockIdx.x - c_first);
            if (tid == 0) {
                all = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) all += sm.fsum[w];
                a.run_stats[place] = make_float2(top, all);
            }
            if (tid < k) a.run_keys[place * k + tid] = sm.cand[tid];
            run = 0;
            m = -INFINITY;
            sum = 0.0f;
            if (!arrive_last(a.row_count + row, 1, n_runs, &sm.last)) continue;
            // -------------------------------------------------------- row
            const uint64_t* rw = a.run_keys + (size_t)row * n_tiles * k;
            const int total = n_runs * k;
            for (int e = tid; e < total; e += kThreads) sm.all[e] = __ldcg(rw + e);
            __syncthreads();
            if (warp == 0) {
                // a lower bound of the row's k-th key: the smallest of every run's ceil(k / runs)-th
                const int m = min(k, (k + n_runs - 1) / n_runs);
                uint64_t b = ~0ull;
                if (lane < n_runs) b = sm.all[lane * k + m - 1];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t w = __shfl_xor_sync(0xffffffffu, b, o);
                    b = w < b ? w : b;
                }
                if (lane == 0) {
                    sm.tau = b;
                    sm.n_cand = 0;
                }
                // log-sum-exp over the runs, one a lane
                const float2 st = lane < n_runs ? __ldcg(a.run_stats + (size_t)row * n_tiles + lane) : make_float2(-INFINITY, 0.0f);
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
        } else {
            // a finished hypothesis: the CTA that has its last tile speaks for it
            if (tile != n_tiles - 1) continue;
            if (tid < k) {
                a.row_keys[(size_t)row * k + tid] = tid == 0 ? score_key((double)base) : 0ull;
                a.row_tokens[(size_t)row * k + tid] = a.end_token;
            }
        }
        // ---------------------------------------------------------------- request
        const int group = row / a.n_beams;
        if (!arrive_last(a.group_count + group, 1, a.n_beams, &sm.last)) continue;
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
        __syncthreads();
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
    a.run_keys = reinterpret_cast<uint64_t*>(p);
    p += rows * tiles * n_out * 8;
    a.run_stats = reinterpret_cast<float2*>(p);
    p += rows * tiles * 8;
    a.row_keys = reinterpret_cast<uint64_t*>(p);
    p += rows * n_out * 8;
    a.row_tokens = reinterpret_cast<int32_t*>(p);
    a.vocab = vocab; a.n_beams = n_beams; a.k = n_out; a.end_token = end_token;
    a.n_tiles = tiles; a.n_rows = (int)rows;
    // a CTA a tile while there are no more than fit at once (four an SM), else even shares of them
    const int sms = va::device_sm_count();
    const long long units = (long long)rows * tiles, most = 4ll * (sms > 0 ? sms : 148);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)(units < most ? units : most)), dim3(va::smp::kThreads), 0, (cudaStream_t)stream);
    return va::paged::launched(format == VA_LOGITS_BF16
                                   ? cudaLaunchKernelEx(&cfg, va::beam::beam_select_kernel<true>, a)
                                   : cudaLaunchKernelEx(&cfg, va::beam::beam_select_kernel<false>, a));
}

}  // extern "C"
