// va_beam_select: beam search's selection over beams and vocabulary.
//
// One launch, three levels.  The (row, 8,192-logit tile) units of the rows that are not finished are dealt evenly to
// four CTAs an SM; a run is a CTA's consecutive tiles of one row.  A CTA reads a tile's logits once (the next two
// tiles' are on their way into L2), and keeps them as they are in memory:
//   sums        every thread keeps its own maximum m and sum of exp(l - m) over the run
//   candidates  the run's k best keys at the last ranking, sorted in shared memory, and the candidates since.  The first
//               tile collects against a lower bound of its k-th logit, as the sampler does; later ones only the logits
//               above the k-th at the last ranking (their indices are higher, so equal ones lose).  A ranking comes
//               with the first tile, the last, and when more than 64 keys wait; a tile without one costs one barrier.
// The last run of a row to arrive merges the runs: log-sum-exp in 64 bits, the row's k best keys and their scores in
// 64 bits.  The last row of a request merges the hypotheses.  Every order is fixed by the keys and by the deal, so the
// arrivals' order changes nothing.
// Bytes: the logits once; what a run hands on (k keys) is a thousandth of that.  32 x 8 x 151,669 bf16 logits, 38 of the
// 256 rows finished (66 MB), take 37.2 us: the tiles' instructions bound it (0.6 us a tile and SM), then the start and
// the merges, which are chains of round trips (5 us and 7 us).  On the way: a 64-bit key for every logit 117 us, a
// ranking for every tile 50 us, finished rows in the deal 50 us, a division for every tile and 32 keys kept in registers
// for the equal logits' sake 39 us; a list for every warp, which needs no barriers but eight times the insertions,
// 67 us; then, where four CTAs an SM took 36.9 us, three 37.2 us, and the next tile's loads before the barrier 38.3 us
// (36.5 us with three CTAs).
// 1 x 4 x 160,000 logits, one row finished: 10.8 us, all of it such chains.
#include <cuda_bf16.h>
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
constexpr int kHold = 64;                                             // keys that wait for a ranking
constexpr int kDirect = 256;                                          // keys that are ranked without a bound first
constexpr int kMaskWords = (kMaxRows + 31) / 32;

struct BeamSmem {
    uint64_t cand[kMaxMerge];   // run: its best at the last ranking, then the candidates since; row and request: what is ranked
    uint64_t best[2][kMaxK];    // run: the best of a ranking, in turn
    int count[3];               // run: candidates of a tile, in turn
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
    uint32_t live[kMaskWords];  // rows that are not finished
    int live_before[kWarps], row0, n_live;
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
    constexpr int kWords = kPerThread * kBytes / 4;               // a thread's part of a tile, in 32-bit words
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_tiles = a.n_tiles, k = a.k;
    auto row_at = [&](int row) { return static_cast<const unsigned char*>(a.logits) + (size_t)row * a.stride * kBytes; };
    auto prefetch = [&](int row, int tile) {      // into L2
        if (tid == 0) {
            const int first = tile * kTileLogits, n = min(kTileLogits, a.vocab - first) * kBytes & ~15;
            if (n > 0) ptx::bulk_prefetch_l2(row_at(row) + (size_t)first * kBytes, (uint32_t)n);
        }
    };
    // where CTA `cta` of `ctas` begins in `units` >= ctas units; those behind the last have none
    auto begin_of = [](unsigned units, unsigned ctas, unsigned cta) { return cta < ctas ? (int)(units * cta / ctas) : (int)units; };
    ptx::griddep_launch_dependents();
    {   // pulled into L2 before the dependency resolves, as in the sampler
        const int u = begin_of((unsigned)a.n_rows * n_tiles, gridDim.x, blockIdx.x);
        prefetch(u / n_tiles, u % n_tiles);
    }
    ptx::griddep_wait();
    // The rows that are not finished, and this CTA's share of their (row, tile) units (at most 2^20, by fewer than 2^11
    // CTAs), in order: u0 .. u1 - 1, beginning in row row0, which is number u0 / n_tiles of them.
    int n_live = a.n_rows, row = 0, next = 0;
    if (a.finished) {
        for (int r0 = warp * 32; r0 < a.n_rows; r0 += kThreads) {
            const bool here = r0 + lane < a.n_rows && __ldcg(a.finished + r0 + lane) == 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, here);
            if (lane == 0) sm.live[r0 / 32] = bits;
        }
        __syncthreads();
        // words w0 .. w0 + per - 1 of a thread, and the live rows before them
        const int words = (a.n_rows + 31) / 32, per = (words + kThreads - 1) / kThreads, w0 = tid * per;
        int mine = 0;
        for (int w = w0; w < min(w0 + per, words); ++w) mine += __popc(sm.live[w]);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += t;
        }
        if (lane == 31) sm.live_before[warp] = upto;
        __syncthreads();
        n_live = 0;
        int before = upto - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? sm.live_before[w] : 0;
            n_live += sm.live_before[w];
        }
        const unsigned units = (unsigned)n_live * n_tiles;
        int target = begin_of(units, min(gridDim.x, units), blockIdx.x) / n_tiles - before;
        if (target >= 0 && target < mine)
            for (int w = w0;; ++w) {
                const int here = __popc(sm.live[w]);
                if (target < here) {
                    sm.row0 = w * 32 + (int)__fns(sm.live[w], 0u, target + 1);
                    break;
                }
                target -= here;
            }
        __syncthreads();
        row = sm.row0;
    }
    const unsigned units = (unsigned)n_live * n_tiles, ctas = min(gridDim.x, units);      // a unit each at least
    const int u0 = begin_of(units, ctas, blockIdx.x), u1 = begin_of(units, ctas, blockIdx.x + 1);
    if (!a.finished) row = u0 / n_tiles;
    // the live row after one
    auto row_after = [&](int row) {
        if (!a.finished) return row + 1;
        int w = (row + 1) / 32;
        const int words = (a.n_rows + 31) / 32;
        if (w >= words) return a.n_rows;
        uint32_t bits = sm.live[w] & (0xFFFFFFFFu << ((row + 1) & 31));
        while (bits == 0u && ++w < words) bits = sm.live[w];
        return bits == 0u ? a.n_rows : w * 32 + __ffs(bits) - 1;
    };
    const float l2e = 1.4426950408889634f, lowest = __uint_as_float(kBf16 ? 0xFF7F0000u : 0xFF7FFFFFu);
    int run = 0;                            // tiles of the run so far
    int held = 0, turn = 0, counter = 0;    // keys in cand; which of the two best, of the three counters is next
    float tau = 0.0f;                       // candidates are at least this
    if (tid < 2 * kMaxK) sm.best[tid / kMaxK][tid % kMaxK] = 0ull;
    float m = -INFINITY, sum = 0.0f;        // this thread's maximum of them, and its sum of exp(l - m)
    int number = u0 / n_tiles, tile = u0 - number * n_tiles;       // the tile at hand: of which live row, which of it
    if (u0 < u1) {
        next = row_after(row);
        if (u0 + 1 < u1) prefetch(tile + 1 < n_tiles ? row : next, tile + 1 < n_tiles ? tile + 1 : 0);
    }
    // then, for the finished rows of this CTA (u >= u1), their only candidate
    int ended = blockIdx.x;
    for (int u = u0;; ++u, ++tile) {
        const bool done = u >= u1;
        if (done) {
            if (!a.finished) break;
            while (ended < a.n_rows && (sm.live[ended / 32] >> (ended & 31) & 1u)) ended += gridDim.x;
            if (ended >= a.n_rows) break;
            row = ended;
            ended += gridDim.x;
        } else if (tile == n_tiles) {
            tile = 0;
            ++number;
            row = next;
            next = row_after(row);
        }
        const unsigned char* src = row_at(row);
        if (!done) {
            const int first = tile * kTileLogits;
            if (u + 2 < u1) {       // the tile after the next
                const bool over = tile + 2 >= n_tiles;
                const int then = over ? tile + 2 - n_tiles : tile + 2;
                if (then < n_tiles) prefetch(over ? next : row, then);
            }
            // -------------------------------------------------------- tile
            uint32_t w[kWords];          // as they are in memory
            const int n_in = min(kTileLogits, a.vocab - first);
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const int at = (i * kThreads + tid) * kVec;
                if (at + kVec <= n_in) {
                    const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)(first + at) * kBytes));
                    w[4 * i] = raw.x;
                    w[4 * i + 1] = raw.y;
                    w[4 * i + 2] = raw.z;
                    w[4 * i + 3] = raw.w;
                } else {   // the row's end: entry by entry, -inf behind it
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (kBf16) {
                            const uint16_t* e = reinterpret_cast<const uint16_t*>(src) + first;
                            const int x = at + 2 * c;
                            const uint32_t lo = x < n_in ? e[x] : 0xFF80u, hi = x + 1 < n_in ? e[x + 1] : 0xFF80u;
                            w[4 * i + c] = lo | hi << 16;
                        } else {
                            const int x = at + c;
                            w[4 * i + c] = x < n_in ? reinterpret_cast<const uint32_t*>(src)[first + x] : 0xFF800000u;
                        }
                    }
                }
            }
            // a NaN is no candidate: -inf; the thread's largest
            float mine = -INFINITY;
            if (kBf16) {
                const __nv_bfloat162 low = __floats2bfloat162_rn(-INFINITY, -INFINITY);
                __nv_bfloat162 top = low;
#pragma unroll
                for (int c = 0; c < kWords; ++c) {
                    const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[c]), low);
                    w[c] = *reinterpret_cast<const uint32_t*>(&x);
                    top = __hmax2(top, x);
                }
                mine = fmaxf(__low2float(top), __high2float(top));
            } else {
#pragma unroll
                for (int c = 0; c < kWords; ++c) {
                    const float x = fmaxf(__uint_as_float(w[c]), -INFINITY);
                    w[c] = __float_as_uint(x);
                    mine = fmaxf(mine, x);
                }
            }
            auto f = [&](int e) {        // the thread's logit e
                return __uint_as_float(kBf16 ? ((e & 1) ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16) : w[e]);
            };
            auto place_of = [&](int e) { return first + ((e / kVec) * kThreads + tid) * kVec + e % kVec; };
            // sums of 2^((l - m) log2 e): subtracted first, because one rounding of m log2 e would stay in the whole sum
            // (4e-5 for a largest logit of 720), and in the row's scores with it.  +inf: its logits share the probability.
            if (mine > -INFINITY) {
                const float up = fmaxf(m, mine);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                if (up < INFINITY) {
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) part[e & 3] += ptx::ex2((f(e) - up) * l2e);
                } else {
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) part[e & 3] += f(e) == up ? 1.0f : 0.0f;
                }
                const float add = (part[0] + part[1]) + (part[2] + part[3]);
                sum = (m == up ? sum : (m == -INFINITY ? 0.0f : sum * ptx::ex2((m - up) * l2e))) + add;
                m = up;
            }
            if (run == 0) {
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
                if (tid == 0) sm.count[counter] = 0;
                __syncthreads();
                uint32_t least = sm.wmin[0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) least = min(least, sm.wmin[w]);
                if (full_warps == 0) least = 0u;
                tau = least > ord_bits(-INFINITY) ? ord_to_float(least) : lowest;
                held = 0;
            }
            // candidates behind those that wait: a warp's take consecutive places.  The tile's counter is cleared two
            // barriers before its use, and read before the next barrier.
            const int mine_is = counter;
            counter = counter == 2 ? 0 : counter + 1;
            if (tid == 0) sm.count[counter] = 0;
            if (__any_sync(0xffffffffu, mine >= tau)) {
                // bit b: in bf16 half b / 16 of word b % 16, else word b
                unsigned bits = 0;
                if (kBf16) {
                    const __nv_bfloat162 bound = __float2bfloat162_rn(tau);      // (tau is one of them)
#pragma unroll
                    for (int c = 0; c < kWords; ++c)
                        bits |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[c]), bound) & (0x10001u << c);
                } else {
#pragma unroll
                    for (int c = 0; c < kWords; ++c) bits |= __uint_as_float(w[c]) >= tau ? 1u << c : 0u;
                }
                const int cnt = __popc(bits);
                int incl = cnt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += t;
                }
                int slot = 0;
                if (lane == 31) slot = atomicAdd(&sm.count[mine_is], incl);
                slot = held + __shfl_sync(0xffffffffu, slot, 31) + incl - cnt;
                for (unsigned rest = bits; rest != 0; rest &= rest - 1) {   // the values are read again (few are)
                    const int b = __ffs(rest) - 1, at = place_of(kBf16 ? 2 * (b & 15) + (b >> 4) : b);
                    const float x = kBf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(src)[at] << 16)
                                          : reinterpret_cast<const float*>(src)[at];
                    if (slot < kMaxMerge) sm.cand[slot] = make_key(x, at);
                    ++slot;
                }
            }
            __syncthreads();
            int n = held + sm.count[mine_is];
            if (n > kMaxMerge) {
                // many equal logits at the bound: the tile's k best by k rounds of block-wide maximum
                uint64_t taken = ~0ull;
                for (int r = 0; r < k; ++r) {
                    uint64_t best = 0;
#pragma unroll
                    for (int c = 0; c < kWords; ++c) asm volatile("" : "+r"(w[c]));     // no 32 keys kept over the rounds
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) {
                        const uint64_t kv = f(e) >= tau ? make_key(f(e), place_of(e)) : 0ull;
                        best = kv < taken && kv > best ? kv : best;
                    }
                    best = block_max_u64(best, sm.red);
                    if (tid == 0) sm.cand[held + r] = best;
                    taken = best;
                }
                n = held + k;
                __syncthreads();
            }
            const bool ends = tile + 1 == n_tiles || u + 1 == u1;
            if (run == 0 || n > kHold || ends) {
                // rank by counting: a key goes to the place of the number of larger ones, if that is below k
                if (tid < k) sm.best[turn ^ 1][tid] = 0ull;
                for (int c = tid; c < n; c += kThreads) {
                    const uint64_t kc = sm.cand[c];
                    int rank = 0;
#pragma unroll 8
                    for (int o = 0; o < n; ++o) rank += sm.cand[o] > kc;
                    if (rank < k && kc != 0ull) sm.best[turn][rank] = kc;
                }
                __syncthreads();
                if (tid < k) sm.cand[tid] = sm.best[turn][tid];
                const uint64_t kth = sm.best[turn][k - 1];
                // the next larger value of the logits' type
                tau = kth != 0ull ? ord_to_float((uint32_t)(kth >> 32) + (kBf16 ? 0x10000u : 1u)) : lowest;
                held = k;
                turn ^= 1;
            } else {
                held = n;
            }
            ++run;
            if (!ends) continue;
            // -------------------------------------------------------- the run's end
            const int c_first = (int)(((unsigned)(number * n_tiles + 1) * ctas - 1u) / units);
            const int c_last = (int)(((unsigned)((number + 1) * n_tiles) * ctas - 1u) / units);
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
            if (tid < k) a.run_keys[place * k + tid] = sm.best[turn ^ 1][tid];
            run = 0;
            m = -INFINITY;
            sum = 0.0f;
            if (!arrive_last(a.row_count + row, 1, n_runs, &sm.last)) continue;
            // -------------------------------------------------------- row
            const uint64_t* rw = a.run_keys + (size_t)row * n_tiles * k;
            const int total = n_runs * k;
            const bool direct = total <= kDirect;
            uint64_t* keys = direct ? sm.cand : sm.all;
            for (int e = tid; e < total; e += kThreads) keys[e] = __ldcg(rw + e);
            if (tid < kMaxK) sm.top[tid] = 0ull;
            __syncthreads();
            if (warp == kWarps - 1) {
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
            } else if (warp == 0 && !direct) {
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
            }
            int nc = total;
            if (!direct) {
                __syncthreads();
                const uint64_t lb = sm.tau;
                for (int e = tid; e < total; e += kThreads) {
                    const uint64_t kv = sm.all[e];
                    if (kv >= lb && kv != 0ull) sm.cand[atomicAdd(&sm.n_cand, 1)] = kv;
                }
                __syncthreads();
                nc = sm.n_cand;
            }
            for (int c = tid; c < nc; c += kThreads) {
                const uint64_t kc = sm.cand[c];
                int rank = 0;
#pragma unroll 8
                for (int o = 0; o < nc; ++o) rank += sm.cand[o] > kc;
                if (rank < k && kc != 0ull) sm.top[rank] = kc;
            }
            __syncthreads();
            if (tid < k) {
                const uint64_t kv = sm.top[tid];
                uint64_t sk = 0ull;
                if (kv != 0ull) {
                    const double l = (double)ord_to_float((uint32_t)(kv >> 32));
                    const double above = l == sm.max ? 0.0 : l - sm.max;
                    sk = score_key((double)__ldcg(a.scores + row) + (above - sm.log_sum));
                }
                a.row_keys[(size_t)row * k + tid] = sk;
                a.row_tokens[(size_t)row * k + tid] = key_index(kv);
            }
        } else {
            // a finished hypothesis
            if (tid < k) {
                a.row_keys[(size_t)row * k + tid] = tid == 0 ? score_key((double)__ldcg(a.scores + row)) : 0ull;
                a.row_tokens[(size_t)row * k + tid] = a.end_token;
            }
        }
        // ---------------------------------------------------------------- request
        const int group = row / a.n_beams;
        if (!arrive_last(a.group_count + group, 1, a.n_beams, &sm.last)) continue;
        const int total = a.n_beams * k;
        const size_t at = (size_t)group * total;
        const bool direct = total <= kDirect;
        uint64_t* keys = direct ? sm.cand : sm.all;
        if (tid == 0) sm.n_cand = 0;
        __syncthreads();
        int mine = 0;
        for (int e = tid; e < total; e += kThreads) {
            keys[e] = __ldcg(a.row_keys + at + e);
            sm.tok[e] = __ldcg(a.row_tokens + at + e);
            if (direct) {
                sm.who[e] = (int16_t)e;
                mine += keys[e] != 0ull;
            }
        }
        if (direct && mine) atomicAdd(&sm.n_cand, mine);
        __syncthreads();
        if (!direct) {
            if (warp == 0) {   // a lower bound of the k-th score: the smallest of every hypothesis' ceil(k / beams)-th
                const int m = (k + a.n_beams - 1) / a.n_beams;
                uint64_t b = lane < a.n_beams ? sm.all[lane * k + m - 1] : ~0ull;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t w = __shfl_xor_sync(0xffffffffu, b, o);
                    b = w < b ? w : b;
                }
                if (lane == 0) sm.tau = b;
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
        }
        // nc candidates among the `in` keys: larger ones first, of equal ones the earlier (its hypothesis, then its order)
        const int nc = sm.n_cand, in = direct ? total : nc;
        const size_t out = (size_t)group * k;
        for (int c = tid; c < in; c += kThreads) {
            const uint64_t kc = sm.cand[c];
            const int e = sm.who[c];
            if (kc == 0ull) continue;
            int rank = 0;
#pragma unroll 8
            for (int o = 0; o < in; ++o) rank += (int)(sm.cand[o] > kc) | ((int)(sm.cand[o] == kc) & (int)(sm.who[o] < e));
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
    const size_t rows = (size_t)n_groups * n_beams;
    if (rows > 1 && (row_stride < vocab || row_stride % (format == VA_LOGITS_BF16 ? 8 : 4) != 0)) return VA_INVALID_ARG;
    if (finished && (end_token < 0 || end_token >= vocab)) return VA_INVALID_ARG;
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
