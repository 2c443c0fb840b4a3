// The split kernel of verify_attn_paged_b8 for many (row, query head) pairs a KV head: tcgen05.
//
// From 17 pairs on, mma.sync would widen each code once per 24 pairs and its products alone would take as long as the
// loads; here every code is widened once, and the products run beside the other work.  Tiles are 128 keys (two pages)
// with keys as the matrix rows: S^T[128 keys x NC pairs] = K Q^T and O^T[128 dimensions x NC pairs] += V^T P^T, f16
// operands in shared memory (exact for both code formats), f32 accumulators in TMEM, S double-buffered.
//   producer   pages' codes and scales into a ring by bulk copies
//   wideners   four warps for K, four for V, from codes to swizzled f16: a page's codes are in registers before their
//              place is free (K's when the scores of the tile before are done, V's two when the products of the tile
//              before the last are)
//   issuer     one thread: the scores of tile i + 1 before the products of tile i
//   scales     one warp: a tile's scales, and the largest V scale
//   softmax    four warps for every 16 pairs, a key a thread: as in paged_attn.cuh (base 2, a reference that is
//              raised when a score passes it by 8, V's scales relative to the largest so far), with one reference a
//              pair for the whole CTA, so that a segment leaves one sum and nothing is joined inside the CTA.  The
//              warps agree on each tile whether to raise; raising rescales the accumulator in TMEM.
// Bound by the softmax warps: 1.6 us for a tile of 128 keys at 48 pairs, 2.9 us where a reference is raised; and by
// what a segment costs once (7.5 us until the first scores, 3 us for its sums).  Measured:
// 48 pairs of one sequence of 192K, E4M3, one KV head 37.1 us, 30 pairs of 32 sequences in a window of 4,096, INT8, two KV
// heads 36.2 us.  (Eight softmax warps, and wideners that took K and V in turn, took 2.2 and 1.6 us more.)
#pragma once

#include "paged_exact.cuh"
#include "paged_plan.cuh"

namespace va {
namespace paged {
namespace tcg {

constexpr int kMaxSoftWarps = 16, kWideWarps = 8;
constexpr int kKeys = 128;                         // keys of a tile
constexpr uint32_t kHalf = kKeys * 128;            // one half of the dimensions of a tile in f16
constexpr uint32_t kOffK = 0, kOffV = 2 * kHalf, kOffP = 6 * kHalf;   // one K buffer, two of V
constexpr uint32_t kPBytes = kKeys * 128;          // a tile's weights: a key a row of 64 pairs
constexpr uint32_t kOffQ = kOffP + kPBytes;        // P and Q together hold NC x 128 floats at a segment's end
constexpr uint32_t kTmemCols = 256, kColS = 0, kColO = 128;   // S at 0 and 64

struct Misc {
    Plan plan;
    alignas(16) float ring_scale[6][8];            // a page's K scales, then its V scales
    alignas(16) float scale[4][16];                // a tile's: K (two pages), V
    alignas(16) float2 fz[kMaxSoftWarps][16];      // per softmax warp and pair of its own: factor and kShift - reference
    float ref[kMaxSoftWarps][16];
    float red[4][kMaxCols], vmax[4];
    alignas(8) uint64_t raw_full[6], raw_empty[6];
    uint64_t k_ready, v_ready[2], s_full[2], s_free[2], p_ready[2], pv_done[2], q_ready, o_done, o_free, vote[2], join, drain;
    int prow[kMaxCols];                            // positions of the pairs' rows
    int ring_ok[6], ok[4];
    alignas(16) unsigned char flag[2][kMaxSoftWarps];
    uint32_t tmem;
    int abort, far;                                // far: the CTA has met V scales far apart
    Share share;
    alignas(16) float2 ub[kMaxSoftWarps][16];      // raising: what comes off a pair's exponents, its sums' factor
};

// Softmax warps: four for every 16 pairs.  Registers a thread at launch (kThreads of them, one CTA an SM), then of the
// softmax warps, the wideners and the last group (producer, issuer, scales and one that waits):
//   NC 32  640 threads x 96 = 256 x 120 + 256 x 72 + 128 x 96
//   NC 48  768 threads x 80 = 384 x  88 + 256 x 72 + 128 x 72
//   NC 64  896 threads x 72 = 512 x  72 + 256 x 64 + 128 x 88
template <int NC>
struct Shape {
    static constexpr int NH = 16;                      // pairs of a softmax warp: one TMEM load's columns
    static constexpr int kSoftWarps = 4 * NC / NH;
    static constexpr int kThreads = 32 * (kSoftWarps + kWideWarps + 4);
    static constexpr int kSoftRegs = NC == 32 ? 120 : (NC == 48 ? 88 : 72), kWideRegs = NC == 64 ? 64 : 72;
    static constexpr int kLaunchRegs = NC == 32 ? 96 : (NC == 48 ? 80 : 72);
    static constexpr int kLastRegs = NC == 32 ? 96 : (NC == 48 ? 72 : 88);
    static constexpr uint32_t kOffRing = kOffQ + NC * 256u;
    static constexpr int kFit = (int)((227u * 1024u - 1024u - kOffRing - sizeof(Misc)) / kTileBytes);
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr int kBytes = 1024 + (int)kOffRing + kStages * kTileBytes + (int)sizeof(Misc);
    static_assert(kStages >= 4, "two tiles of pages");
    static_assert(kSoftWarps >= kExactWarps && sizeof(ExactSmem) <= kOffRing, "exact_segments' warps and place");
};

__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Sixteen codes to sixteen f16 values, in order.
template <bool kInt8>
__device__ __forceinline__ void widen16(const uint4& c, uint4& lo, uint4& hi) {
    uint32_t r[8];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kInt8) {
            const uint32_t u = w[i] ^ 0x80808080u;
            const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
            uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
            const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
            r[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
            r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
        } else {
            asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
                : "=r"(r[2 * i]), "=r"(r[2 * i + 1]) : "r"(w[i]));
        }
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

template <bool kInt8, int NC>
__global__ void __launch_bounds__(Shape<NC>::kThreads, 1)
    attn_paged_tc_kernel(const AttnPagedArgs a) {
    using S = Shape<NC>;
    constexpr int NR = S::kStages, NH = S::NH, kSoftWarps = S::kSoftWarps, kThreads = S::kThreads;
    constexpr int kIssuer = kSoftWarps + kWideWarps;       // then the producer's and the scales' warp
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = base + S::kOffRing;
    Misc& ms = *reinterpret_cast<Misc*>(ring + NR * kTileBytes);
    const uint32_t base_s = ptx::smem_u32(base);
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    volatile int* abort = &ms.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < NR; ++s) {
            ptx::mbar_init(bar(ms.raw_full[s]), 1);
            ptx::mbar_init(bar(ms.raw_empty[s]), kWideWarps + 1);
        }
        ptx::mbar_init(bar(ms.k_ready), kWideWarps / 2 + 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar(ms.v_ready[s]), kWideWarps / 2);
            ptx::mbar_init(bar(ms.s_full[s]), 1);
            ptx::mbar_init(bar(ms.s_free[s]), kSoftWarps);
            ptx::mbar_init(bar(ms.p_ready[s]), kSoftWarps);
            ptx::mbar_init(bar(ms.pv_done[s]), 1);
            ptx::mbar_init(bar(ms.vote[s]), kSoftWarps);
        }
        ptx::mbar_init(bar(ms.q_ready), kSoftWarps);
        ptx::mbar_init(bar(ms.o_done), 1);
        ptx::mbar_init(bar(ms.o_free), kSoftWarps);
        ptx::mbar_init(bar(ms.join), kSoftWarps);
        ptx::mbar_init(bar(ms.drain), 1);
        ptx::mbar_init_fence();
        ms.abort = ms.far = 0;
        for (int s = 0; s < 2; ++s) *reinterpret_cast<uint4*>(ms.flag[s]) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int status = 0;
    const Share share = make_plan<kThreads>(ms.plan, a);
    if ((int)blockIdx.x >= share.n_ctas || share.n == 0) return;
    if (tid == 0) ms.share = share;
    if (warp == 0) ptx::tmem_alloc(ptx::smem_u32(&ms.tmem), kTmemCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const int heads = a.n_kv * a.group, n_cols = a.n_rows * a.group;

    if (warp >= kIssuer) {
    if constexpr (S::kLastRegs < S::kLaunchRegs) ptx::set_max_regs_dec<S::kLastRegs>();
    if constexpr (S::kLastRegs > S::kLaunchRegs) ptx::set_max_regs_inc<S::kLastRegs>();
    if (warp == kIssuer + 1) {
        // ------------------------------------------------------------ producer: 32 pages looked up at once
        int last = -1;
        bool given_up = false;
        for (int i0 = 0; i0 < share.n && !given_up; i0 += 32) {
            int row = -1;
            if (i0 + lane < share.n) row = tile_row(ms.plan, a, share.c0 + i0 + lane, status);
            for (int l = 0; l < 32 && i0 + l < share.n; ++l) {
                const int i = i0 + l, s = i % NR, use = i / NR, r = __shfl_sync(0xffffffffu, row, l);
                if (use > 0 && !warp_wait(bar(ms.raw_empty[s]), (use - 1) & 1, abort, status)) {
                    given_up = true;
                    break;
                }
                const uint32_t full = bar(ms.raw_full[s]);
                if (lane == 0) {
                    ms.ring_ok[s] = r >= 0;
                    if (r >= 0) ptx::mbar_arrive_expect_tx(full, kTileBytes + 32);
                    else ptx::mbar_arrive(full);
                }
                __syncwarp();
                if (r >= 0) {
                    if (lane < 2)
                        ptx::bulk_load(ptx::smem_u32(ring + s * kTileBytes) + lane * kHeadBytes,
                                       (lane ? a.v_codes : a.k_codes) + (size_t)r * kHeadBytes, kHeadBytes, full);
                    else if (lane < 4)
                        ptx::bulk_load(ptx::smem_u32(ms.ring_scale[s]) + 16 * (lane - 2),
                                       (lane == 2 ? a.k_scale : a.v_scale) + (size_t)r * kBlocks, 16, full);
                }
                last = i;
            }
        }
        // no CTA ends with copies under way, even if the others gave up
        for (int i = max(0, last + 1 - NR); i <= last; ++i)
            ptx::mbar_wait(bar(ms.raw_full[i % NR]), (i / NR) & 1, nullptr, kWaitNs);
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ issuer (one lane)
        if (lane == 0) {
            bool ok = true;
            auto wait = [&](uint64_t& b, int phase) {
                if (ok && !ptx::mbar_wait(bar(b), phase & 1, abort, kWaitNs)) {
                    if (!*abort) status |= VA_DEV_TIMEOUT;
                    *abort = 1;
                    ok = false;
                }
                return ok;
            };
            constexpr uint32_t id_s = idesc_f16(kKeys, NC, 0, 0);     // K and Q: the dimension contiguous
            constexpr uint32_t id_o = idesc_f16(kKeys, NC, 1, 1);     // V^T and P^T: dimensions and pairs contiguous
            auto scores = [&](int t) {
                if (!wait(ms.k_ready, t) || (t >= 2 && !wait(ms.s_free[t & 1], (t >> 1) - 1))) return;
                ptx::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t h = k >> 2, off = (k & 3) * 32;
                    ptx::mma_bf16(tmem + kColS + (t & 1) * 64, ptx::smem_desc(base_s + kOffK + h * kHalf + off, 0, 1024),
                                  ptx::smem_desc(base_s + kOffQ + h * NC * 128u + off, 0, 1024), id_s, k > 0);
                }
                ptx::mma_commit(bar(ms.s_full[t & 1]));
            };
            auto products = [&](int t, int n_keys16, bool first, bool end, int seg) {
                if (!wait(ms.v_ready[t & 1], t >> 1) || !wait(ms.p_ready[t & 1], t >> 1)) return;
                if (first && seg > 0 && !wait(ms.o_free, seg - 1)) return;
                ptx::tc_fence_after();
                for (int k = 0; k < n_keys16; ++k)
                    ptx::mma_bf16(tmem + kColO, ptx::smem_desc(base_s + kOffV + (t & 1) * 2 * kHalf + k * 2048, kHalf, 1024),
                                  ptx::smem_desc(base_s + kOffP + k * 2048, 8192, 1024), id_o,
                                  !first || k > 0);
                ptx::mma_commit(bar(ms.pv_done[t & 1]));
                if (end) ptx::mma_commit(bar(ms.o_done));
            };
            Walk walk(share);
            int t = 0;
            while (ok && walk.next(ms.plan, a, share.n)) {
                const int pages = walk.end - walk.begin, n = (pages + 1) / 2;
                if (wait(ms.q_ready, walk.seg)) {
                    scores(t);
                    for (int i = 0; i < n && ok; ++i) {
                        if (i + 1 < n) scores(t + i + 1);
                        products(t + i, 2 * i + 1 < pages ? 8 : 4, i == 0, i + 1 == n, walk.seg);
                    }
                }
                t += n;
            }
            ptx::mma_commit(bar(ms.drain));      // all products done before TMEM is given back
            ptx::mbar_wait(bar(ms.drain), 0, nullptr, kWaitNs);
        }
        __syncwarp();
    } else if (warp == kIssuer + 2) {
        // ------------------------------------------------------------ the tiles' scales, and their largest V scales
        Walk walk(share);
        int t = 0;
        bool ok = true;
        while (ok && walk.next(ms.plan, a, share.n)) {
            const int from = seen_from(walk.len, walk.live, a.window);
            uint32_t highest = 0u, lowest = 0x7F800000u;     // of the segment's V scales, this lane's
            for (int p0 = walk.begin; p0 < walk.end; p0 += 2, ++t) {
                const int n_pages = min(2, walk.end - p0), key0 = (walk.page0 + p0 - walk.begin) * kPage;
                float sc[2] = {0.0f, 0.0f}, vmax = 0.0f;
                int good = 0;
                for (int hp = 0; hp < n_pages && ok; ++hp) {
                    const int s = (p0 + hp) % NR;
                    if (!(ok = warp_wait(bar(ms.raw_full[s]), ((p0 + hp) / NR) & 1, abort, status))) break;
                    const bool page_ok = ms.ring_ok[s] != 0;
                    if (lane < 8) sc[hp] = ms.ring_scale[s][lane];
                    // V's of blocks that no row sees are 0
                    const int at = key0 + hp * kPage + kBlock * (lane & 3);
                    const bool in = page_ok && lane >= 4 && lane < 8 && at < walk.len && at + kBlock > from;
                    if (!in && lane >= 4) sc[hp] = 0.0f;
                    // (positive floats order like their bits)
                    vmax = fmaxf(vmax, __uint_as_float(__reduce_max_sync(0xffffffffu, in ? __float_as_uint(sc[hp]) : 0u)));
                    good |= page_ok ? 1 << hp : 0;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(ms.raw_empty[s]));
                }
                // with the keys of this tile, not before (the barrier counts both)
                if (!ok || (t > 0 && !(ok = warp_wait(bar(ms.s_full[(t - 1) & 1]), ((t - 1) >> 1) & 1, abort, status)))) break;
                if (lane < 8) {
                    ms.scale[t & 3][(lane & 4) * 2 + (lane & 3)] = sc[0];
                    ms.scale[t & 3][(lane & 4) * 2 + 4 + (lane & 3)] = sc[1];
                }
                if (lane == 0) {
                    ms.vmax[t & 3] = vmax;
                    ms.ok[t & 3] = good;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(ms.k_ready));
#pragma unroll
                for (int hp = 0; hp < 2; ++hp) {
                    const uint32_t s = lane >= 4 ? __float_as_uint(sc[hp]) : 0u;
                    highest = max(highest, s);
                    lowest = min(lowest, s == 0u ? 0x7F800000u : s);
                }
            }
            highest = __reduce_max_sync(0xffffffffu, highest);
            lowest = __reduce_min_sync(0xffffffffu, lowest);
            if (lane == 0 && __uint_as_float(highest) > fminf(kFar / 2 * __uint_as_float(lowest), kHuge / 2)) ms.far = 1;
        }
    }
    } else if (warp >= kSoftWarps) {
        ptx::set_max_regs_dec<S::kWideRegs>();
        // ------------------------------------------------------------ wideners: four warps for K, four for V
        // Thread (row r0, r0 + 16, .. of each page; 16-byte chunk c).  A page's codes are in registers before the place
        // they go to is free, so the page is given back early.
        const int wt = (tid - 32 * kSoftWarps) & 127;
        const bool is_v = warp >= kSoftWarps + kWideWarps / 2;
        const int c = wt & 7, r0 = wt >> 3;
        const int first = 2 * (c & 3) + (c >> 2), second = first ^ 1;   // order of the two f16 chunks: no bank twice
        Walk walk(share);
        int t = 0;
        bool ok = true;
        while (ok && walk.next(ms.plan, a, share.n)) {
            for (int p0 = walk.begin; p0 < walk.end; p0 += 2, ++t) {
                const int n_pages = min(2, walk.end - p0);
                const int key0 = (walk.page0 + p0 - walk.begin) * kPage;
                uint4 x[2][4];
#pragma unroll
                for (int hp = 0; hp < 2; ++hp)
                    if (hp < n_pages && ok) {
                        const int s = (p0 + hp) % NR;
                        ok = warp_wait(bar(ms.raw_full[s]), ((p0 + hp) / NR) & 1, abort, status);
                        const unsigned char* src = ring + s * kTileBytes + (is_v ? kHeadBytes : 0) + r0 * kD + c * 16;
#pragma unroll
                        for (int u = 0; u < 4; ++u) x[hp][u] = *reinterpret_cast<const uint4*>(src + 16 * u * kD);
                        // (what lies past the sequence or in no page may be NaN, and would stay it with weight 0)
                        const int in = ms.ring_ok[s] != 0 ? walk.len - key0 - hp * kPage - r0 : 0;
                        if (is_v && in < kPage) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (16 * u >= in) x[hp][u] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(ms.raw_empty[s]));
                    }
                // K's buffer is free once the scores of the tile before are done, V's once the products of the one
                // before that are
                if (ok && t > (is_v ? 1 : 0))
                    ok = warp_wait(is_v ? bar(ms.pv_done[t & 1]) : bar(ms.s_full[(t - 1) & 1]),
                                   (is_v ? (t >> 1) - 1 : (t - 1) >> 1) & 1, abort, status);
                if (!ok) break;
                unsigned char* to = base + (is_v ? kOffV + (t & 1) * 2 * kHalf : kOffK) + (c >> 2) * kHalf + r0 * 128;
#pragma unroll
                for (int hp = 0; hp < 2; ++hp)
                    if (hp < n_pages) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint4 y[2];
                            widen16<kInt8>(x[hp][u], y[0], y[1]);
                            unsigned char* dst = to + (hp * kPage + 16 * u) * 128;
                            *reinterpret_cast<uint4*>(dst + ((first ^ (r0 & 7)) * 16)) = c & 4 ? y[1] : y[0];
                            *reinterpret_cast<uint4*>(dst + ((second ^ (r0 & 7)) * 16)) = c & 4 ? y[0] : y[1];
                        }
                    }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(is_v ? bar(ms.v_ready[t & 1]) : bar(ms.k_ready));
            }
        }
    } else {
        if constexpr (S::kSoftRegs > S::kLaunchRegs) ptx::set_max_regs_inc<S::kSoftRegs>();
        // ------------------------------------------------------------ softmax: key (or dimension) 32 q + lane, pairs n0..
        const int q = warp & 3, n0 = (warp >> 2) * NH, me = 32 * q + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        float2* fz = ms.fz[warp];
        float* ref = ms.ref[warp];
        Walk walk(share);
        int t = 0, joins = 0;
        bool ok = true;
        // All of these warps have come here (with a limit).
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(ms.join));
            ok = warp_wait(bar(ms.join), joins++ & 1, abort, status);
            return ok;
        };
        while (ok && walk.next(ms.plan, a, share.n)) {
            const int b = walk.b, h = walk.h, len = walk.len, live = walk.live, pages = walk.end - walk.begin;
            auto row_of = [&](int c) {      // of pair c, in q, out and out_lse
                return ((size_t)b * a.n_rows + ms.plan.col_row[c]) * heads + h * a.group + ms.plan.col_head[c];
            };
            // Q, each row brought to f16's upper range by a power of two, a row a warp at a time
            uint2 raws[NC / kSoftWarps];
#pragma unroll
            for (int k = 0; k < NC / kSoftWarps; ++k) {
                const int c = warp + k * kSoftWarps;
                raws[k] = make_uint2(0u, 0u);
                if (c < n_cols && ms.plan.col_row[c] < live)
                    raws[k] = __ldg(reinterpret_cast<const uint2*>(a.q + row_of(c) * kD) + lane);
            }
#pragma unroll
            for (int k = 0; k < NC / kSoftWarps; ++k) {
                const int c = warp + k * kSoftWarps;
                const uint2 raw = raws[k];
                const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(raw.x & 0x7FFFu, (raw.x >> 16) & 0x7FFFu),
                                                                        max(raw.y & 0x7FFFu, (raw.y >> 16) & 0x7FFFu)));
                const int up = min(max(268 - (int)(top >> 7), 1), 253);
                const float by = __uint_as_float((uint32_t)up << 23);
                const __half2 x = __floats2half2_rn(__uint_as_float(raw.x << 16) * by, __uint_as_float(raw.x & 0xFFFF0000u) * by);
                const __half2 y = __floats2half2_rn(__uint_as_float(raw.y << 16) * by, __uint_as_float(raw.y & 0xFFFF0000u) * by);
                // dimensions 4 lane .. 4 lane + 3: half lane / 16, chunk (lane % 16) / 2, 8 bytes of it
                unsigned char* dst = base + kOffQ + (lane >> 4) * (NC * 128) + c * 128 +
                                     ((((lane & 15) >> 1) ^ (c & 7)) * 16) + (lane & 1) * 8;
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
                if (lane == 0) ms.prow[c] = len - live + (c < n_cols ? min((int)ms.plan.col_row[c], live - 1) : live - 1);
                if (lane < 4)
                    ms.fz[4 * (c / NH) + lane][c % NH] = make_float2(__uint_as_float((uint32_t)(254 - up) << 23) * a.scale_log2, kShift);
            }
            if (lane < NH) ref[lane] = kNoScore;
            ptx::fence_proxy_async_smem();
            if (!meet()) break;                        // (the factors are written by other warps)
            if (lane == 0) ptx::mbar_arrive(bar(ms.q_ready));
            float l[NH];
#pragma unroll
            for (int c = 0; c < NH; ++c) l[c] = 0.0f;
            float R = 0.0f, inv_r = 0.0f;
            bool all_set = false;
            const int n_tiles = (pages + 1) / 2;
            for (int i = 0; i < n_tiles; ++i, ++t) {
                if (!(ok = warp_wait(bar(ms.s_full[t & 1]), (t >> 1) & 1, abort, status))) break;
                ptx::tc_fence_after();
                float y[NH];
                ptx::tmem_ld16_wait(tl + kColS + (t & 1) * 64 + n0, y);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(ms.s_free[t & 1]));
                // this thread's key, its block's scales
                const int hp = me >> 6, key0 = (walk.page0 + 2 * i) * kPage, key = key0 + me;
                const float* sc = ms.scale[t & 3];
                const int n_here = 2 * i + 1 < pages ? 2 : 1;
                const bool seen = hp < n_here && ((ms.ok[t & 3] >> hp) & 1) && key < len;
                const float ks = seen ? sc[me >> 4] : 0.0f, vs = seen ? sc[8 + (me >> 4)] : 0.0f;
                const bool edge = key0 + n_here * kPage - 1 > len - live || (a.window > 0 && key0 < len - a.window);
                float high = -INFINITY;
                const float4* fz4 = reinterpret_cast<const float4*>(fz);
#pragma unroll
                for (int c = 0; c < NH; c += 2) {
                    const float4 w = fz4[c / 2];
                    y[c] = fmaf(y[c], w.x * ks, w.y);
                    y[c + 1] = fmaf(y[c + 1], w.z * ks, w.w);
                    high = fmaxf(high, fmaxf(y[c], y[c + 1]));
                }
                if (!seen) {
                    high = -INFINITY;
#pragma unroll
                    for (int c = 0; c < NH; ++c) y[c] = -INFINITY;
                }
                if (edge) {
#pragma unroll
                    for (int c = 0; c < NH; ++c) {
                        const int p = ms.prow[n0 + c];
                        if (key > p || (a.window > 0 && key <= p - a.window)) y[c] = -INFINITY;
                    }
                }
                // (edge: the keys that a pair does not see may raise too, which does no harm)
                const float vmax = ms.vmax[t & 3];
                bool raise = i == 0 || vmax > R || high > kShift + kLazy;
                if (!all_set) {      // a pair without a reference takes any score as a reason
#pragma unroll
                    for (int c = 0; c < NH; ++c) raise = raise || (y[c] > -INFINITY && ref[c] == kNoScore);
                }
                raise = __any_sync(0xffffffffu, raise);
                if (lane == 0) {
                    ms.flag[t & 1][warp] = raise;
                    ptx::mbar_arrive(bar(ms.vote[t & 1]));
                }
                if (!(ok = warp_wait(bar(ms.vote[t & 1]), (t >> 1) & 1, abort, status))) break;
                const volatile unsigned long long* flags = reinterpret_cast<const volatile unsigned long long*>(ms.flag[t & 1]);
                if ((flags[0] | flags[1]) != 0) {
                    // columns' maxima over the tile's keys, by warp, then over the four warps that share them
#pragma unroll
                    for (int c = 0; c < NH; ++c) {
                        const float top = ptx::redux_max(y[c]);
                        if (lane == 0) ms.red[q][n0 + c] = top;
                    }
                    if (!meet()) break;
                    float r_by = 1.0f;
                    if (vmax > R) {
                        const uint32_t next = (__float_as_uint(vmax) + 0x7FFFFFu) & 0x7F800000u;
                        const float up = __uint_as_float(min(next, 0x7F000000u));
                        r_by = R / up;
                        R = up;
                        inv_r = 1.0f / up;
                    }
                    float o[NH];
                    if (i > 0) {
                        if (!(ok = warp_wait(bar(ms.pv_done[(t - 1) & 1]), ((t - 1) >> 1) & 1, abort, status))) break;
                        ptx::tc_fence_after();
                        ptx::tmem_ld16_wait(tl + kColO + n0, o);
                    }
                    // lane c finds pair n0 + c's new reference
                    if (lane < NH) {
                        const int c = n0 + lane;
                        const float now = fmaxf(fmaxf(ms.red[0][c], ms.red[1][c]), fmaxf(ms.red[2][c], ms.red[3][c]));
                        const float was = ref[lane];
                        const bool none_yet = was == kNoScore;
                        const float up = now == -INFINITY ? 0.0f : (none_yet ? now - kShift : fmaxf(now - kShift, 0.0f));
                        ms.ub[warp][lane] = make_float2(up, none_yet ? 1.0f : ptx::ex2(-up));
                        if (now > -INFINITY) {
                            const float m = (none_yet ? 0.0f : was) + up;
                            ref[lane] = m;
                            fz[lane].y = kShift - m;
                        }
                    }
                    __syncwarp();
                    const float4* ub = reinterpret_cast<const float4*>(ms.ub[warp]);
#pragma unroll
                    for (int c = 0; c < NH; c += 2) {
                        const float4 w = ub[c / 2];
                        y[c] -= w.x;
                        l[c] *= w.y;
                        y[c + 1] -= w.z;
                        l[c + 1] *= w.w;
                        if (i > 0) {
                            o[c] *= w.y * r_by;
                            o[c + 1] *= w.w * r_by;
                        }
                    }
                    if (i > 0) {
                        ptx::tmem_st16(tl + kColO + n0, o);
                        ptx::tmem_wait_st();
                    }
                    ptx::tc_fence_before();
                    all_set = __all_sync(0xffffffffu, lane >= NH || ref[lane] != kNoScore);
                }
                // weights into P, which the products of the tile before have left
                if (t > 0 && !(ok = warp_wait(bar(ms.pv_done[(t - 1) & 1]), ((t - 1) >> 1) & 1, abort, status))) break;
                const float r = vs * inv_r;
                unsigned char* dst = base + kOffP + me * 128;
#pragma unroll
                for (int c8 = 0; c8 < NH / 8; ++c8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = ptx::ex2(y[8 * c8 + 2 * e]), p1 = ptx::ex2(y[8 * c8 + 2 * e + 1]);
                        l[8 * c8 + 2 * e] += p0;
                        l[8 * c8 + 2 * e + 1] += p1;
                        const __half2 x = __floats2half2_rn(p0 * r, p1 * r);
                        w[e] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                    *reinterpret_cast<uint4*>(dst + (((n0 / 8 + c8) ^ (me & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(ms.p_ready[t & 1]));
            }
            if (!ok) break;
            // -------------------------------------------------------- the segment's sums
            // In rolled loops over shared memory (P's and Q's place, now free): this runs once or twice in a CTA, from a
            // cold instruction cache, where a line of code costs as much as a load.
            if (!(ok = warp_wait(bar(ms.o_done), walk.seg & 1, abort, status))) break;
            ptx::tc_fence_after();
            float* stage = reinterpret_cast<float*>(base + kOffP);
#pragma unroll
            for (int c = 0; c < NH; ++c) stage[(n0 + c) * kKeys + me] = l[c];
            float o[NH];
            ptx::tmem_ld16_wait(tl + kColO + n0, o);
            ptx::tc_fence_before();
            if (!meet()) break;
            if (lane == 0) ptx::mbar_arrive(bar(ms.o_free));
            const size_t part = (size_t)(2 * blockIdx.x + (walk.begin == 0 ? 0 : 1)) * kMaxCols;
#pragma unroll 1
            for (int c = warp; c < NC; c += kSoftWarps) {
                const float4 v = reinterpret_cast<const float4*>(stage + c * kKeys)[lane];
                float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float at = ms.ref[4 * (c / NH)][c % NH];
                const float m = at == kNoScore ? -INFINITY : at - kShift;
                float by = 0.0f;
                if (c < n_cols && ms.plan.col_row[c] < live) {
                    by = R;
                    if (walk.whole) {
                        const int head = h * a.group + ms.plan.col_head[c];
                        const Finish fin = finish(m, sum, a.sink, head);
                        by *= fin.by;
                        if (lane == 0 && a.out_lse) a.out_lse[row_of(c)] = fin.lse;
                    } else if (lane == 0) {
                        a.part_ml[part + c] = make_float2(m, sum);
                    }
                }
                if (lane == 0) ms.red[0][c] = by;
            }
            if (!meet()) break;
#pragma unroll
            for (int c = 0; c < NH; ++c) stage[(n0 + c) * kKeys + me] = o[c];
            if (!meet()) break;
#pragma unroll 1
            for (int c = warp; c < NC; c += kSoftWarps) {
                if (c >= n_cols || ms.plan.col_row[c] >= live) continue;
                float4 v = reinterpret_cast<const float4*>(stage + c * kKeys)[lane];
                const float by = ms.red[0][c];
                v.x *= by;
                v.y *= by;
                v.z *= by;
                v.w *= by;
                if (walk.whole)
                    store_row(a.out + row_of(c) * kD + 4 * lane, v);
                else
                    reinterpret_cast<float4*>(a.part_o + (part + c) * kD)[lane] = v;
            }
            if (!meet()) break;
        }
    }
    if (status && a.dev_status) atomicOr(a.dev_status, status);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    // segments whose V scales lie far apart, again
    if (__builtin_expect(ms.far != 0, 0) && warp < kExactWarps) {
        const Share again = ms.share;
        exact_segments<kInt8>(a, ms.plan, again, *reinterpret_cast<ExactSmem*>(base));
    }
}

template <bool kInt8, int NC>
cudaError_t launch(const AttnPagedArgs& a, cudaStream_t stream) {
    const cudaError_t e = ensure_smem_attr((const void*)attn_paged_tc_kernel<kInt8, NC>, Shape<NC>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    pdl_config(&cfg, attr, dim3((unsigned)a.n_ctas), dim3(Shape<NC>::kThreads), Shape<NC>::kBytes, stream);
    return cudaLaunchKernelEx(&cfg, attn_paged_tc_kernel<kInt8, NC>, a);
}

}  // namespace tcg
}  // namespace paged
}  // namespace va
