// The split kernel of prompt_attn_paged_b8 and verify_attn_shared_b8: tcgen05, 256 pairs x 128 keys a step.
//
// S[128 pairs x 128 keys] = Q K^T and O[128 pairs x 128 dimensions] += P V, twice a step (two times 128 pairs share the
// keys), f16 operands (exact for both code formats), f32 accumulators in TMEM: S at columns 0 and 128, O at 256 and 384.
// A pair is a TMEM lane and a thread of the softmax warps, which needs no other thread for its maximum and its sum.
//   softmax    two times four warps: S from TMEM, P back into the columns of S as f16, from where the products read it.
//              Base 2.  Key j's weight carries its value's scale as a term of the exponent, p_j = 2^(s_j + log2 v_j - m + 3), so
//              that P's range does not depend on the scales; the sum of weights divides it out again, 16 keys at a time.
//              m is raised when an exponent passes it by 12; then the row of O is rescaled.
//   wideners   eight warps, each a block (16 keys) of a tile's K and one of its V: codes from global memory to registers a tile
//              ahead, then to swizzled f16 in shared memory
//   scales     one warp: the tiles' scales
//   issuer     one thread: the products of a tile, then the scores of the next, for each 128 pairs in turn, so that one
//              set of softmax warps works while the tensor cores serve the other.  Units of up to 128 pairs leave the second
//              set idle in prompts; in shared calls, most of whose units they are, the two sets take their tiles in turn, each
//              with a sum of its own, and the first joins them (8 x 8 slots of 4K 42.7 -> 38.5 us; in prompts the issuer's
//              longer code cost more than that gave, turns 221 -> 238 us)
// What bounds it: a step takes 3,780 cycles, of which the products are 2,048 and no other unit is busier: each 128 pairs' chain of
// scores, exponents, weights and products, of which tensor memory holds two and no third.  A chunk of 2K rows at 128K (6 heads
// on 1, INT8) takes 644 us, 1.27 PFLOP/s, a 16K prompt 353 us (its join 12 of them).  Widening, done again for every unit that
// reads a page, is 101 us of the chunk.  Tried and slower: pairs of CTAs that widen half the keys each
// (chunk 925 us, handoffs through the cluster); 16 softmax warps with half a pair's keys a thread (699); no wideners, the
// softmax warps widening (999); no search for a maximum but a check of the sums (779).
// Registers: 640 threads x 96 at launch = 256 x 144 (softmax) + 384 x 64.  The code is kept short (one copy of each step, in
// rolled loops): a launch runs from a cold instruction cache, and small calls are bound by that.
#pragma once

#include <cuda_fp16.h>

#include "prompt_plan.cuh"

namespace va {
namespace paged {
namespace pr {

constexpr int kWide0 = 8, kScales = 16, kIssuer = 17;
constexpr int kSoftRegs = 144, kOtherRegs = 64;
static_assert(kThreads == 640 && 256 * kSoftRegs + 384 * kOtherRegs <= kThreads * 96, "what the launch has, for 20 warps");
constexpr uint32_t kHalf = kKeys * 128;                       // 64 dimensions of 128 rows in f16
constexpr uint32_t kOffQ = 0, kOffK = 4 * kHalf, kOffV = 8 * kHalf;   // two of each
constexpr uint32_t kOffMisc = 12 * kHalf;
constexpr uint32_t kColO = 256, kTmemCols = 512;
// p = 2^(t - m + kUnit); m is raised when a t passes it by kRaise, so that p stays below 2^15.  A product of weight and value
// scale of 2^-17 of the row's largest or less loses digits in f16 (it is rounded to 2^-28 of that).  Raising costs the row of
// O once through the registers: with 2^6 and 8, where a third of the tiles of a long history with some large keys raised in one
// of 128 rows, a chunk of 2K rows at 128K took 958 us, with 2^3 and 12 873.
constexpr float kUnit = 3.0f, kRaise = 12.0f;
// Exponents from where on t - m is taken of the rounded t: their own roundings, and those of m + log2 v, would come to more
// than a twentieth, and soon to more than f16 holds.
constexpr float kFar = 262144.0f;
// 2^-60, which smaller scales of values (and zeros, whose keys weigh in the sum) count as: from an inverse of 2^80 on sums
// of weights could pass fp32.  And 2^60, beyond which weights may be lost next to smaller scales.  Both are told of.
constexpr float kLeastScale = 8.673617e-19f, kMostScale = 1.152921505e18f;

template <bool kShared>
struct Misc {
    Deal<kShared> deal;
    alignas(16) float scale[4][kKeys / 32][8];                // a tile's blocks in twos: K's scales, log2 of V's, their inverses, -
    int bad[4][2];                                            // is a page of the tile none?
    alignas(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_ready[2], q_ready[2], o_full[2], lent, gave, drain;
    float fac[128];                                           // where both sets take the same pairs: what the first knows of their queries,
    float2 ml[128];                                           // and what the second has of them in the end
    Place place[kThreads / 32], to;                           // of each warp's next segment; the CTA's end
    uint32_t tmem;
    int abort;
};
template <bool kShared>
constexpr int smem_bytes() {
    return 1024 + (int)kOffMisc + (int)sizeof(Misc<kShared>);
}
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory");

__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Eight codes to eight f16 values, in order.
template <bool kInt8>
__device__ __forceinline__ uint4 widen8(const uint32_t c0, const uint32_t c1) {
    uint32_t r[4];
    const uint32_t w[2] = {c0, c1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
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
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Two f32 to f16, the first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Where a pair of a segment lies: its row in q, out and out_lse (rows of 128), the keys that it sees.
struct Pair {
    size_t row;
    int lo, hi;                  // hi < 0: there is no such pair
};
template <bool kShared>
__device__ __forceinline__ Pair pair_of(const Args& a, const Deal<kShared>& d, int e, int h, const Unit& u, int k, int i) {
    Pair p;
    p.row = 0;
    p.lo = 0;
    p.hi = -1;
    if (i >= u.pairs) return p;
    const int n = k * kPairs + i, heads = a.n_kv * a.group;
    int b, r = a.by_group.quotient(n), g = n - r * a.group;
    if constexpr (!kShared) {
        b = e;
        p.row = (size_t)d.extra[b] + r;
    } else {
        const int gr = a.by_slots.quotient(e), j = e - gr * (a.share + 1);
        b = gr * a.share + j - 1;
        if (j == 0) {
            const int slot = a.by_rows.quotient(r);
            b = gr * a.share + slot;
            r -= slot * a.n_rows;
        }
        p.row = (size_t)b * a.n_rows + r;
    }
    if (r >= d.live[b]) return p;
    p.row = p.row * heads + h * a.group + g;
    const int at = d.len[b] - d.live[b] + r;
    p.hi = min(at, (int)min((long long)(u.first + u.n) * kPage - 1, 0x7FFFFFFFll));
    p.lo = a.window > 0 ? max(0, at - a.window + 1) : 0;
    return p;
}

// The pages of a unit, 32 entries of the table at a time, one a lane.
struct Pages {
    const int32_t* table;                        // the unit's entries
    int n, held, entry;                          // entries held .. held + 31 (-1: none, -2: past the unit's end)
    __device__ __forceinline__ Pages(const int32_t* first, int n_pages) : table(first), n(n_pages), held(-32), entry(-2) {}
    __device__ __forceinline__ int at(int i, int pool) {
        const int lane = threadIdx.x & 31;
        if (i >= held + 32) {
            held = i & ~1;                       // (whole tiles)
            entry = -2;
            if (held + lane < n) {
                entry = __ldcg(table + held + lane);
                if (entry < 0 || entry >= pool) entry = -1;
            }
        }
        return __shfl_sync(0xffffffffu, entry, i - held);
    }
};

// A widener's work: block `block` of every tile's K and V.  Lane (row r0, r0 + 4, .. of a block; 16 codes, which are the chunks
// 2 c and 2 c + 1 of a row's half in f16): the eight lanes that shared memory serves at a time write four chunks each of two
// rows next to each other, whose swizzled places differ in the lowest bit.
template <bool kInt8, bool kShared>
__device__ __forceinline__ void widen_tiles(const Args& a, Misc<kShared>& ms, unsigned char* base, int block, int& status) {
    const Deal<kShared>& deal = ms.deal;
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    volatile int* abort = &ms.abort;
    const int lane = threadIdx.x & 31, c = lane & 3, half = (lane >> 3) & 1, r0 = ((lane >> 2) & 1) + 2 * (lane >> 4);
    unsigned char* const to0 = base + half * kHalf + (block * kBlock + r0) * 128;
    const int lane_at = (block % kBlocks * kBlock + r0) * kD + half * 64 + c * 16, hp = block / kBlocks;
    Segment seg;
    int tt = 0;
    while (seg.next(deal, a, ms.place[kWide0 + block], ms.to, true)) {
        const int row = deal.table_row(a, seg.e);
        // positions from the lane's first row of the segment's first tile on that the sequence has
        int in = min(kShared && a.by_slots.rest(seg.e) == 0 ? 0x7FFFFFFF : deal.len[row] - seg.u.first * kPage, seg.u.n * kPage) -
                 2 * seg.t0 * kPage - block * kBlock - r0;
        Pages pages(a.table + (size_t)row * a.max_pages + seg.u.first, seg.u.n);
        const int h = seg.h, n = seg.t1 - seg.t0;
        int i = 2 * seg.t0 + hp, page = -1;
        uint4 x[2][4];
        // (what lies past the sequence or in no page may be NaN, and would stay it with weight 0)
        auto load = [&](uint4 (&y)[4], const uint8_t* codes) {
            const uint8_t* src = codes + ((size_t)max(page, 0) * a.n_kv + h) * kHeadBytes + lane_at;
            const int here = page < 0 ? 0 : in;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = make_uint4(0u, 0u, 0u, 0u);
                if (4 * r < here) y[r] = __ldcg(reinterpret_cast<const uint4*>(src + 4 * r * kD));
            }
        };
        auto widen = [&](const uint4 (&y)[4], unsigned char* to, uint64_t& full) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int place = (2 * c) ^ ((r0 + 4 * r) & 7);
                *reinterpret_cast<uint4*>(to + 4 * r * 128 + place * 16) = widen8<kInt8>(y[r].x, y[r].y);
                *reinterpret_cast<uint4*>(to + 4 * r * 128 + (place ^ 1) * 16) = widen8<kInt8>(y[r].z, y[r].w);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(full));
        };
        // t: the tile that is widened; the one behind it is loaded meanwhile
#pragma unroll 1
        for (int t = -1; t < n; ++t) {
            const int stage = tt & 1, turn = tt >> 1;
            if (t >= 0) {
                if (turn > 0 && !warp_wait(bar(ms.k_empty[stage]), (turn - 1) & 1, abort, status)) return;
                widen(x[0], to0 + kOffK + stage * 2 * kHalf, ms.k_full[stage]);
            }
            const bool more = t + 1 < n;
            if (more) {
                page = pages.at(i, a.n_pages);
                i += 2;
                load(x[0], a.k_codes);
            }
            if (t >= 0) {
                if (turn > 0 && !warp_wait(bar(ms.v_empty[stage]), (turn - 1) & 1, abort, status)) return;
                widen(x[1], to0 + kOffV + stage * 2 * kHalf, ms.v_full[stage]);
                ++tt;
            }
            if (more) {
                load(x[1], a.v_codes);
                in -= kKeys;
            }
        }
    }
}

// The scales' warp: lanes 0..7 K's of a tile's eight blocks, 8..15 V's.
template <bool kShared>
__device__ __forceinline__ void tile_scales(const Args& a, Misc<kShared>& ms, int& status) {
    const Deal<kShared>& deal = ms.deal;
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    volatile int* abort = &ms.abort;
    const int lane = threadIdx.x & 31, block = lane & 7, kv = (lane >> 3) & 1;
    Segment seg;
    int tt = 0;
    while (seg.next(deal, a, ms.place[kScales], ms.to, true)) {
        const int row = deal.table_row(a, seg.e);
        const int end = min(kShared && a.by_slots.rest(seg.e) == 0 ? 0x7FFFFFFF : deal.len[row] - seg.u.first * kPage, seg.u.n * kPage);
        Pages pages(a.table + (size_t)row * a.max_pages + seg.u.first, seg.u.n);
        const float* const scales = (kv ? a.v_scale : a.k_scale) + (size_t)seg.h * kBlocks + block % kBlocks;
#pragma unroll 1
        for (int t = seg.t0; t < seg.t1; ++t, ++tt) {
            const int p0 = pages.at(2 * t, a.n_pages), p1 = pages.at(2 * t + 1, a.n_pages), page = block < kBlocks ? p0 : p1;
            float x = 0.0f;
            // (blocks past the sequence's end may hold anything)
            if (lane < 16 && page >= 0 && 2 * t * kPage + block * kBlock < end) x = __ldcg(scales + (size_t)page * a.n_kv * kBlocks);
            if (p0 == -1 || p1 == -1) status |= VA_DEV_BAD_PAGE;
            if (tt >= 2 && !warp_wait(bar(ms.k_empty[tt & 1]), ((tt >> 1) - 1) & 1, abort, status)) return;
            if (lane < 16) {
                const float least = fmaxf(x, kLeastScale);
                float* const to = &ms.scale[tt & 3][block >> 1][block & 1];
                to[2 * kv] = kv ? log2f(least) : x;
                if (kv) to[4] = 1.0f / least;
                if (kv && x != 0.0f && !(x >= kLeastScale && x <= kMostScale)) status |= VA_DEV_VALUE_SCALE;
                if (lane < 8 && block % kBlocks == 0) ms.bad[tt & 3][block / kBlocks] = page == -1;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(ms.k_full[tt & 1]));
        }
    }
}

template <bool kInt8, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) prompt_tc_kernel(const Args a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    Misc<kShared>& ms = *reinterpret_cast<Misc<kShared>*>(base + kOffMisc);
    const uint32_t base_s = ptx::smem_u32(base);
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    volatile int* abort = &ms.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar(ms.k_full[s]), 9);
            ptx::mbar_init(bar(ms.k_empty[s]), 1);
            ptx::mbar_init(bar(ms.v_full[s]), 8);
            ptx::mbar_init(bar(ms.v_empty[s]), 1);
            ptx::mbar_init(bar(ms.s_full[s]), 1);
            ptx::mbar_init(bar(ms.p_half[s]), 4);
            ptx::mbar_init(bar(ms.p_ready[s]), 4);
            ptx::mbar_init(bar(ms.q_ready[s]), 4);
            ptx::mbar_init(bar(ms.o_full[s]), 1);
        }
        ptx::mbar_init(bar(ms.lent), 4);
        ptx::mbar_init(bar(ms.gave), 4);
        ptx::mbar_init(bar(ms.drain), 1);
        ptx::mbar_init_fence();
        ms.abort = 0;
        ms.deal.rows = 0;
    }
    __syncthreads();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (warp == 2) ptx::tmem_alloc(ptx::smem_u32(&ms.tmem), kTmemCols);
    ms.deal.make(a, ms.place[0], ms.to);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const Deal<kShared>& deal = ms.deal;
    if (tid < kThreads / 32 && tid > 0) ms.place[tid] = ms.place[0];
    __syncthreads();
    int status = 0;

    if (warp >= kWide0) {
    ptx::set_max_regs_dec<kOtherRegs>();        // (whole groups of four warps)
    if (warp == kIssuer) {
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
            constexpr uint32_t id_s = idesc_f16(128, kKeys, 0, 0), id_o = idesc_f16(128, kD, 0, 1);
            int n_seg[2] = {0, 0}, n_p[2] = {0, 0}, turns = 0, tt = 0, goes_on = 0;
            int4 begun = make_int4(-1, 0, 0, 0);
            // (descriptors count in 16 bytes; nothing carries out of their 14 bits of address)
            const uint64_t desc_q = ptx::smem_desc(base_s + kOffQ, 0, 1024), desc_k = ptx::smem_desc(base_s + kOffK, 0, 1024);
            const uint64_t desc_v = ptx::smem_desc(base_s + kOffV, kHalf, 1024);
            constexpr uint32_t kTile16 = 2 * kHalf / 16;
            auto scores = [&](int w, int q, int t) {
                const uint64_t qa = desc_q + q * kTile16, ka = desc_k + (t & 1) * kTile16;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) / 16;
                    ptx::mma_bf16(tmem + w * 128, qa + off, ka + off, id_s, i > 0);
                }
                ptx::mma_commit(bar(ms.s_full[w]));
            };
            Segment seg;
            while (ok && seg.next(deal, a, ms.place[kIssuer], ms.to, false)) {
                const int n = seg.t1 - seg.t0;
                const bool few = seg.u.pairs <= 128;
                if (!seg.first) goes_on = seg.last ? 1 : 2;
                if constexpr (!kShared) {
                    if (seg.first && !seg.last) begun = make_int4(deal.live[seg.e], deal.extra[seg.e], seg.h, seg.k);
                }
                if (kShared && seg.first) {
                    const int blocks = (a.share * a.n_rows * a.group + kPairs - 1) / kPairs;
                    a.first_cta[unit_number(a, blocks, seg.e, seg.h, seg.k)] = seg.last ? -1 : (int)blockIdx.x;
                }
                if constexpr (!kShared) {
                    const int mt = few ? 1 : 2;
                    for (int w = 0; w < mt; ++w)
                        if (!wait(ms.q_ready[w], n_seg[w]++)) break;
                    if (!wait(ms.k_full[tt & 1], tt >> 1)) break;
                    ptx::tc_fence_after();
                    for (int w = 0; w < mt; ++w) scores(w, w, tt);
                    ptx::mma_commit(bar(ms.k_empty[tt & 1]));
                    for (int j = 0; j < n && ok; ++j) {
                        const int t = tt + j;
                        for (int w = 0; w < mt && ok; ++w) {
                            if (w == 0 && !wait(ms.v_full[t & 1], t >> 1)) break;
                            const uint64_t vd = desc_v + (t & 1) * kTile16;
                            auto products = [&](int i0) {
                                ptx::tc_fence_after();
#pragma unroll
                                for (int i = i0; i < i0 + 4; ++i)
                                    ptx::mma_f16_ta(tmem + kColO + w * 128, tmem + w * 128 + 8 * i + 32 * (i >> 2), vd + i * (2048 / 16), id_o,
                                                    j > 0 || i > 4 || i0 == 0);
                            };
                            // (the second half's weights come first)
                            if (!wait(ms.p_half[w], n_p[w])) break;
                            products(4);
                            if (!wait(ms.p_ready[w], n_p[w]++)) break;
                            products(0);
                            if (w == mt - 1) ptx::mma_commit(bar(ms.v_empty[t & 1]));
                            if (j + 1 < n) {
                                if (w == 0) {
                                    if (!wait(ms.k_full[(t + 1) & 1], (t + 1) >> 1)) break;
                                    ptx::tc_fence_after();
                                }
                                scores(w, w, t + 1);
                                if (w == mt - 1) ptx::mma_commit(bar(ms.k_empty[(t + 1) & 1]));
                            } else {
                                ptx::mma_commit(bar(ms.o_full[w]));
                            }
                        }
                    }
                } else {
                    // (rolled: small calls are bound by code that is fetched for the first time)
                    if (!wait(ms.q_ready[0], n_seg[0]++) || (!few && !wait(ms.q_ready[1], n_seg[1]++))) break;
                    if (!wait(ms.k_full[tt & 1], tt >> 1)) break;
                    ptx::tc_fence_after();
                    scores(0, 0, tt);
                    if (!few) scores(1, 1, tt);
                    ptx::mma_commit(bar(ms.k_empty[tt & 1]));
                    if (few && n > 1) {
                        if (!wait(ms.k_full[(tt + 1) & 1], (tt + 1) >> 1)) break;
                        ptx::tc_fence_after();
                        scores(1, 0, tt + 1);
                        ptx::mma_commit(bar(ms.k_empty[(tt + 1) & 1]));
                    }
                    const int next = few ? 2 : 1;        // a set's next tile
                    for (int j = 0; j < n && ok; ++j) {
                        const int t = tt + j;
#pragma unroll 1
                        for (int w = few ? j & 1 : 0; w < (few ? (j & 1) + 1 : 2) && ok; ++w) {
                            const bool first = few || w == 0, last = few || w == 1;     // of the tile's sets
                            if (first && !wait(ms.v_full[t & 1], t >> 1)) break;
                            const uint64_t vd = desc_v + (t & 1) * kTile16;
                            auto products = [&](int i0) {
                                ptx::tc_fence_after();
#pragma unroll
                                for (int i = i0; i < i0 + 4; ++i)
                                    ptx::mma_f16_ta(tmem + kColO + w * 128, tmem + w * 128 + 8 * i + 32 * (i >> 2), vd + i * (2048 / 16), id_o,
                                                    j >= next || i > 4 || i0 == 0);
                            };
                            // (the second half's weights come first)
                            const int turn = turns >> w;
                            turns ^= 1 << w;
                            if (!wait(ms.p_half[w], turn)) break;
                            products(4);
                            if (!wait(ms.p_ready[w], turn)) break;
                            products(0);
                            if (last) ptx::mma_commit(bar(ms.v_empty[t & 1]));
                            if (j + next < n) {
                                const int s = t + next;
                                if (first) {
                                    if (!wait(ms.k_full[s & 1], s >> 1)) break;
                                    ptx::tc_fence_after();
                                }
                                scores(w, few ? 0 : w, s);
                                if (last) ptx::mma_commit(bar(ms.k_empty[s & 1]));
                            } else if (!few || j == n - 1) {
                                ptx::mma_commit(bar(ms.o_full[few ? 0 : w]));
                            }
                        }
                    }
                }
                tt += n;
            }
            a.begun[blockIdx.x] = begun;
            a.goes_on[blockIdx.x] = goes_on;
            ptx::mma_commit(bar(ms.drain));      // all products done before TMEM is given back
            ptx::mbar_wait(bar(ms.drain), 0, nullptr, kWaitNs);
        }
        __syncwarp();
    } else if (warp < kScales) {
        widen_tiles<kInt8>(a, ms, base, warp - kWide0, status);
    } else if (warp == kScales) {
        tile_scales(a, ms, status);
    }
    } else {
        ptx::set_max_regs_inc<kSoftRegs>();
        // ------------------------------------------------------------ softmax: a pair a thread
        const int w = warp >> 2, me = tid & 127;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16), ts = tl + w * 128, to = tl + kColO + w * 128;
        Segment seg;
        int tt = 0, n_s = 0, n_seg = 0, n_both = 0;
        bool ok = true;
        while (ok && seg.next(deal, a, ms.place[warp], ms.to, true)) {
            // up to 128 pairs are the first set's; in shared calls both's, who take their tiles in turn
            const int n = seg.t1 - seg.t0;
            const bool few = seg.u.pairs <= 128, one = kShared && few, both = one && n > 1;
            if (w == 1 && few && !both) {
                tt += n;
                continue;
            }
            const int i0 = few ? 0 : w * 128;    // its pairs begin here in the unit
            const Pair pair = pair_of<kShared>(a, deal, seg.e, seg.h, seg.u, seg.k, i0 + me);
            // Q: whole rows into their places as bf16, then each thread's row brought to f16's upper range by a power of two.
            // (Rows read by their threads cost a tag lookup a lane and load.)
            unsigned char* const mine = base + kOffQ + w * 2 * kHalf + (warp & 3) * 32 * 128;     // the warp's rows
            float fac;
            const int n_rows = min(32, seg.u.pairs - i0 - 32 * (warp & 3));     // (no more in use: the others' rows of S
                                                                                     // and O are never looked at)
            if (one && w == 1) {
                if (!(ok = warp_wait(bar(ms.lent), n_both & 1, abort, status))) break;
                fac = ms.fac[me];
            } else {
#pragma unroll 4
                for (int r0 = 0; r0 < n_rows; r0 += 2) {
                    const int r = r0 + (lane >> 4), c = lane & 15;
                    const bool on = __shfl_sync(0xffffffffu, pair.hi, r) >= 0;
                    const size_t row = ((size_t)__shfl_sync(0xffffffffu, (uint32_t)(pair.row >> 32), r) << 32) |
                                       __shfl_sync(0xffffffffu, (uint32_t)pair.row, r);
                    ptx::copy16(ptx::smem_u32(mine + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) * 16)), a.q + row * kD + 8 * c, on);
                }
                ptx::copies_landed();
                __syncwarp();
                uint32_t top = 0;
                uint4* const x0 = reinterpret_cast<uint4*>(mine + lane * 128);
#pragma unroll 8
                for (int i = 0; i < 16; ++i) {
                    const uint4 x = x0[(i >> 3) * (kHalf / 16) + ((i & 7) ^ (lane & 7))];
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
                }
                top = max(top >> 16, top & 0xFFFFu);
                const int up = min(max(268 - (int)(top >> 7), 1), 253);
                const float by = __uint_as_float((uint32_t)up << 23 | (a.flip & 0x80000000u));
                fac = __uint_as_float((uint32_t)(254 - up) << 23) * a.scale_log2;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    uint4& at = x0[(i >> 3) * (kHalf / 16) + ((i & 7) ^ (lane & 7))];
                    const uint4 x = at;
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = pack_f16(__uint_as_float(in[e] << 16) * by, __uint_as_float(in[e] & 0xFFFF0000u) * by);
                    at = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (both && w == 0) ms.fac[me] = fac;
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0 && !(one && w == 1)) {
                ptx::mbar_arrive(bar(ms.q_ready[w]));
                if (both) ptx::mbar_arrive(bar(ms.lent));
            }
            // (a pair that is none takes part without a mask, its q being 0 or anything)
            const int my_hi = pair.hi >= 0 ? pair.hi : 0x7FFFFFFF, my_lo = pair.lo;
            const int warp_hi = __reduce_min_sync(0xffffffffu, my_hi), warp_lo = __reduce_max_sync(0xffffffffu, my_lo);
            float m = kNoScore, l = 0.0f;
#pragma unroll 1
            for (int j = one ? w : 0; j < n; j += one ? 2 : 1) {
                if (!(ok = warp_wait(bar(ms.s_full[w]), n_s++ & 1, abort, status))) break;
                ptx::tc_fence_after();
                if (n_rows <= 0) {
                    if (lane == 0) {
                        ptx::mbar_arrive(bar(ms.p_half[w]));
                        ptx::mbar_arrive(bar(ms.p_ready[w]));
                    }
                    continue;
                }
                const int slot = (tt + j) & 3;
                const long long key0 = (long long)(seg.u.first + 2 * (seg.t0 + j)) * kPage;
                bool exact = key0 + kKeys - 1 > warp_hi || key0 < warp_lo || (ms.bad[slot][0] | ms.bad[slot][1]) != 0;
                // The weights of 16 keys from their scores: packed, and their sum
                float sum = 0.0f;
                auto weights = [&](const float* x, float k, float plus, float inv, uint32_t* p) {
                    const float2 by = make_float2(k, k), add = make_float2(plus, plus);
                    float2 u, v;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 e = ptx::fma2(make_float2(x[2 * i], x[2 * i + 1]), by, add);
                        const float2 y = make_float2(ptx::ex2(e.x), ptx::ex2(e.y));
                        if (i == 0) u = y;
                        else if (i == 1) v = y;
                        else if (i & 1) v = ptx::add2(v, y);
                        else u = ptx::add2(u, y);
                        p[i] = pack_f16(y.x, y.y);
                    }
                    u = ptx::add2(u, v);
                    sum = fmaf(u.x + u.y, inv, sum);
                };
                auto largest = [&](const float* x) {
                    float y = x[0], z = x[1];
#pragma unroll
                    for (int i = 2; i < 14; i += 4) {
                        y = ptx::max3(y, x[i], x[i + 1]);
                        z = ptx::max3(z, x[i + 2], x[i + 3]);
                    }
                    return fmaxf(z, ptx::max3(y, x[14], x[15]));
                };
                // The largest exponent is known: raises the reference, and the sums with it
                auto refer = [&](float top) {
                    const bool need = top > m + kRaise && pair.hi >= 0;
                    if (__any_sync(0xffffffffu, need)) {
                        const float up = need ? top : m, lower = need ? ptx::ex2(m - up) : 1.0f;
                        m = up;
                        l *= lower;
                        if (j > (one ? 1 : 0)) {
#pragma unroll 1
                            for (int c = 0; c < 128; c += 16) {
                                float o[16];
                                ptx::tmem_ld16_wait(to + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= lower;
                                ptx::tmem_st16(to + c, o);
                            }
                        }
                    }
                    return kUnit - m;
                };
                // P of the second half of the keys, whose products may begin: at the columns of its own scores
                auto half_done = [&]() {
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(ms.p_half[w]));
                };
                const float (*const scale)[8] = ms.scale[slot];
                if (!kShared && !exact) {
                    // 32 keys at a time, the next ones on their way: all for the largest exponent, the second half's weights from
                    // the registers, the first half again for its weights.  (Shared calls have few tiles a CTA and are bound by code
                    // that is fetched for the first time: with this step in the kernel 1 x 32 x 16K took 53 us instead of 49.)
                    float x[32], y[32];
                    uint32_t p[32];
                    auto top_of = [&](const float* s, int b) {
                        const float4 z = *reinterpret_cast<const float4*>(scale[b]);
                        return fmaxf(fmaf(largest(s), z.x * fac, z.z), fmaf(largest(s + 16), z.y * fac, z.w));
                    };
                    float base_m;
                    auto weights_of = [&](const float* s, int b, uint32_t* to_p) {
                        const float4 z = *reinterpret_cast<const float4*>(scale[b]);
                        const float2 inv = *reinterpret_cast<const float2*>(scale[b] + 4);
                        weights(s, z.x * fac, z.z + base_m, inv.x, to_p);
                        weights(s + 16, z.y * fac, z.w + base_m, inv.y, to_p + 8);
                    };
                    ptx::tmem_ld32(ts, x);
                    ptx::tmem_landed(x);
                    ptx::tmem_ld32(ts + 32, y);
                    float top = top_of(x, 0);
                    ptx::tmem_landed(y);
                    ptx::tmem_ld32(ts + 64, x);
                    top = fmaxf(top, top_of(y, 1));
                    ptx::tmem_landed(x);
                    ptx::tmem_ld32(ts + 96, y);
                    top = fmaxf(top, top_of(x, 2));
                    ptx::tmem_landed(y);
                    top = fmaxf(top, top_of(y, 3));
                    exact = __any_sync(0xffffffffu, fabsf(top) >= kFar && pair.hi >= 0);
                    if (!exact) {
                        base_m = refer(top);
                        weights_of(x, 2, p);
                        ptx::tmem_ld32(ts, x);
                        weights_of(y, 3, p + 16);
                        ptx::tmem_st32w(ts + 64, p);
                        half_done();
                        ptx::tmem_landed(x);
                        ptx::tmem_ld32(ts + 32, y);
                        weights_of(x, 0, p);
                        ptx::tmem_landed(y);
                        weights_of(y, 1, p + 16);
                        ptx::tmem_st32w(ts, p);
                    }
                }
                if (kShared || exact) {
                    // the same by halves in a loop: the first for the largest exponent; the second for that, then its weights; the
                    // first again.  Exact: exponents are rounded, masked and compared here, of which no more than the difference
                    // goes on.
                    float s[64], kc[4], plus[4], top = -INFINITY, base_m = 0.0f;
#pragma unroll 1
                    for (int pass = 0; pass < 3; ++pass) {
                        const int h = pass & 1;
                        ptx::tmem_ld32(ts + 64 * h, s);
                        ptx::tmem_ld32(ts + 64 * h + 32, s + 32);
                        ptx::tmem_landed(s);
#pragma unroll
                        for (int b = 0; b < 4; b += 2) {
                            const float4 z = *reinterpret_cast<const float4*>(scale[2 * h + (b >> 1)]);
                            kc[b] = z.x * fac;
                            kc[b + 1] = z.y * fac;
                            plus[b] = z.z;
                            plus[b + 1] = z.w;
                        }
                        if (exact) {
                            const int hi = ms.bad[slot][h] ? -1 : (int)max(min((long long)my_hi - key0, 127ll) - 64 * h, -1ll);
                            const int lo = (int)min(max((long long)my_lo - key0 - 64 * h, 0ll), 64ll);
                            // (a bit a key that is seen)
                            const unsigned long long seen = ((hi >= 63 ? 0ull : 2ull << max(hi, 0)) - 1ull) & (hi < 0 ? 0ull : lo > 63 ? 0ull : ~0ull << lo);
                            const uint32_t bits[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
#pragma unroll
                                for (int i = 16 * b; i < 16 * b + 16; ++i) s[i] = bits[i >> 5] >> (i & 31) & 1u ? fmaf(s[i], kc[b], plus[b]) : -INFINITY;
                                kc[b] = 1.0f;
                                plus[b] = 0.0f;
                            }
                        }
                        if (pass < 2) {
#pragma unroll
                            for (int b = 0; b < 4; ++b) top = fmaxf(top, fmaf(largest(s + 16 * b), kc[b], plus[b]));
                        }
                        if (pass == 0) continue;
                        if (pass == 1) {
                            if (!exact && __any_sync(0xffffffffu, fabsf(top) >= kFar && pair.hi >= 0)) {
                                exact = true;
                                top = -INFINITY;
                                pass = -1;
                                continue;
                            }
                            base_m = refer(top);
                        }
                        uint32_t p[32];
#pragma unroll
                        for (int b = 0; b < 4; ++b) weights(s + 16 * b, kc[b], plus[b] + base_m, scale[2 * h + (b >> 1)][4 + (b & 1)], p + 8 * b);
                        ptx::tmem_st32w(ts + 64 * h, p);
                        if (pass == 1) half_done();
                    }
                }
                l += sum;
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(ms.p_ready[w]));
            }
            tt += n;
            if (!ok) break;
            if (one && w == 1) {
                ms.ml[me] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(ms.gave));
                ++n_both;
                continue;
            }
            if (!(ok = warp_wait(bar(ms.o_full[w]), n_seg++ & 1, abort, status))) break;
            ptx::tc_fence_after();
            float ours = 1.0f, theirs = 0.0f;    // factors of the two sets' sums
            if (both) {
                if (!(ok = warp_wait(bar(ms.gave), n_both++ & 1, abort, status))) break;
                const float2 other = ms.ml[me];
                const float top = fmaxf(m, other.x);
                ours = ptx::ex2(m - top);
                theirs = ptx::ex2(other.x - top);
                l = fmaf(l, ours, other.y * theirs);
                m = top;
            }
            // the row of O: the output, or partial sums; by way of the places of Q, from where a warp writes whole rows
            const float ref = m == kNoScore ? -INFINITY : m - kUnit;
            const bool whole = seg.first && seg.last, out = !kShared && whole;
            float by = 1.0f;
            unsigned char* dst = reinterpret_cast<unsigned char*>(a.out);
            size_t at = pair.row;                // of the pair in there
            if (out) {
                const Finish f = finish(ref, l, a.sink, seg.h * a.group + a.by_group.rest(seg.k * kPairs + i0 + me));
                by = f.by;
                if (pair.hi >= 0 && a.out_lse) a.out_lse[at] = f.lse;
            } else {
                float2* ml = a.part_ml;
                dst = reinterpret_cast<unsigned char*>(a.part_o);
                if (kShared && whole) {
                    ml = a.pair_ml;
                    dst = reinterpret_cast<unsigned char*>(a.pair_o);
                    at += a.by_slots.rest(seg.e) == 0 ? 0 : (size_t)a.n_seqs * a.n_rows * a.n_kv * a.group;
                } else {
                    at = (size_t)(2 * blockIdx.x + (seg.first ? 1 : 0)) * kPairs + i0 + me;
                }
                if (pair.hi >= 0) ml[at] = make_float2(ref, l);
            }
            auto stage = [&](int r, int k) {     // 16 bytes of the warp's 32 rows of 256 (where its rows of Q were)
                return mine + (r >> 4) * kHalf + (r & 15) * 256 + ((k ^ (r & 15)) * 16);
            };
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                // 32 columns: a quarter of a row in bf16, or half of it in fp32
                float o[32];
                ptx::tmem_ld32(to + 32 * c, o);
                ptx::tmem_landed(o);
                if (both) {
                    float z[32];
                    ptx::tmem_ld32(to + 128 + 32 * c, z);
                    ptx::tmem_landed(z);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(o[i], ours, z[i] * theirs);
                }
                const int k0 = out ? 4 * c : 8 * (c & 1);
                if (!out) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(stage(lane, k0 + i)) =
                            make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t z[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * i + 2 * e] * by, o[8 * i + 2 * e + 1] * by);
                            z[e] = *reinterpret_cast<const uint32_t*>(&y);
                        }
                        *reinterpret_cast<uint4*>(stage(lane, k0 + i)) = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                }
                if (c != 3 && (out || c != 1)) continue;
                __syncwarp();
#pragma unroll 4
                for (int r0 = 0; r0 < n_rows; r0 += 2) {
                    const int r = r0 + (lane >> 4), k = lane & 15;
                    const uint4 z = *reinterpret_cast<const uint4*>(stage(r, k));
                    const bool on = __shfl_sync(0xffffffffu, pair.hi, r) >= 0;
                    const size_t row = ((size_t)__shfl_sync(0xffffffffu, (uint32_t)(at >> 32), r) << 32) | __shfl_sync(0xffffffffu, (uint32_t)at, r);
                    if (on) *reinterpret_cast<uint4*>(dst + row * (out ? 256 : 512) + (out || c == 1 ? 0 : 256) + k * 16) = z;
                }
                __syncwarp();
            }
            ptx::tc_fence_before();
        }
    }
    if (status && a.dev_status) atomicOr(a.dev_status, status);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kInt8, bool kShared>
cudaError_t launch(const Args& a, cudaStream_t stream) {
    const cudaError_t e = ensure_smem_attr((const void*)prompt_tc_kernel<kInt8, kShared>, smem_bytes<kShared>());
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    pdl_config(&cfg, attr, dim3((unsigned)a.n_ctas), dim3(kThreads), smem_bytes<kShared>(), stream);
    return cudaLaunchKernelEx(&cfg, prompt_tc_kernel<kInt8, kShared>, a);
}

}  // namespace pr
}  // namespace paged
}  // namespace va
