// The split kernel of verify_attn_paged_b8 for few (row, query head) pairs a KV head (instantiated per format in
// paged_attn_e4m3.cu / paged_attn_int8.cu); paged_plan.cuh has the deal of the batch's tiles over the CTAs.
//
// Inside a CTA four warps feed a ring of pages by TMA and eight consume it: teams of two warps take the tiles in turn,
// each warp half of the page's keys for all pairs, so no barrier joins the warps between tiles.  With keys as the
// matrix rows, S^T = K Q^T and O^T = V^T P^T need as many 8-column tiles as there are pairs / 8: a single token of six
// heads costs one, where queries as matrix rows would cost two.  The codes are widened to f16 in registers (exact for
// both formats) and multiplied by mma.sync: a code is used by so few pairs that its load bounds the call, and tensor
// memory would only add a way through shared memory.
//   Keys are taken in the order 0 5 2 7 4 1 6 3 of each eight: with the 128-byte swizzle of the loads, the 16-byte
//   shared-memory reads of K (two rows a phase) and of V (four rows of even or odd order) then meet no bank twice.
// The softmax is online, in base 2: p = 2^(t - m + 6) with m raised only when a score passes it by 8, so f16 holds
// p <= 2^14 to 11 bits down to 2^-20 of the maximum (and to 2^-31 of it absolutely); sums are fp32.  The blocks' V
// scales go into p relative to R, the largest so far (a power of two), which f16 would not hold by themselves
// (scales that lie far apart: paged_exact.cuh).
// Measured, E4M3, one token of 6 query heads a KV head: 64 sequences of 1 to 16K positions, 8 KV heads (262 MB) 59.0
// us, 4.4 TB/s; 4 sequences of 1K, one KV head 10.9 us, most of it the two launches' and the segments' one-time work.
#pragma once

#include "paged_attn_tc.cuh"
#include "paged_exact.cuh"
#include "paged_plan.cuh"

namespace va {
namespace paged {

constexpr int kConsumers = 8;                 // consumer warps of a CTA
// Three warpgroups of 168 registers a thread at launch (64,512 in all); the consumers' two then hold 232, the
// producer's one 40 (59,392 + 5,120).
constexpr int kAttnThreads = 32 * (kConsumers + 4);
constexpr int kConsumerRegs = 232, kProducerRegs = 40;
constexpr int kTickets = 64;                  // segments that can be open at once in a CTA are fewer
constexpr int kSplit = 2;                     // warps that share a page's blocks
constexpr int kTeams = kConsumers / kSplit;   // a power of two

// ----------------------------------------------------------------------------- fragments
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A word's codes c0..c3 to the f16 pairs (c0, c1), (c2, c3), exactly.  E4M3: two conversions, which issue like any
// integer instruction here (2.2 cycles a warp measured; placing the bits by shifts and masks took seven).  INT8:
// 0x64xx is 1024 + xx, so the biased code (+128) becomes the low byte and 1152 comes off again (taking 1152 sum q off
// a score instead would save the subtractions here, and lose five bits of the score).
template <bool kInt8>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& x, uint32_t& y) {
    if (kInt8) {
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 lo = __hsub2(*reinterpret_cast<__half2*>(&a), bias), hi = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
        x = *reinterpret_cast<const uint32_t*>(&lo);
        y = *reinterpret_cast<const uint32_t*>(&hi);
    } else {
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
            : "=r"(x), "=r"(y) : "r"(w));
    }
}

// A stage's use number `use` has been loaded (bar: its full barrier) or read (its empty barrier): first that the
// use's loads have been issued (*issued > use), because a barrier's parity alone does not tell the use that is
// waited for from the one before the last; then the barrier.
__device__ __forceinline__ bool page_wait(volatile int* issued, int use, uint32_t bar, uint32_t parity, volatile int* abort,
                                          int& status) {
    bool ok = true;
    if (*issued <= use) {
        const uint64_t t0 = ptx::globaltimer_ns();
        while (*issued <= use && ok) ok = !*abort && ptx::globaltimer_ns() - t0 <= kWaitNs;
    }
    if (!__all_sync(0xffffffffu, ok)) {
        if (!*abort) status |= VA_DEV_TIMEOUT;
        __syncwarp();
        *abort = 1;
        return false;
    }
    return warp_wait(bar, parity, abort, status);
}

// ----------------------------------------------------------------------------- shared memory
// RT: 8-pair tiles of a warp; kStages: pages in flight.
template <int RT>
struct Shape {
    static constexpr int kCols = 8 * RT;                                       // pairs
    static constexpr int kSlotFloats = kCols * kD;
    static constexpr int kFixed = kConsumers * (kSlotFloats + 10 * kCols) * 4  // the warps' slots, (m, l) and weights
                                  + (int)sizeof(Plan) + 2048;                  // barriers, tickets, share, alignment
    static constexpr int kFit = (227 * 1024 - 1024 - kFixed) / (kTileBytes + 32);
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr int kBytes = 1024 + kFixed + kStages * (kTileBytes + 32);
    static_assert(kStages >= 4, "the ring needs a few pages");
    static_assert(sizeof(ExactSmem) <= kConsumers * kSlotFloats * 4, "in the slots' place");
    static_assert(sizeof(Plan) % 16 == 0, "the scales behind it are written by bulk copies");
};

template <bool kInt8, int RT>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_paged_kernel(const AttnPagedArgs a, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
    using S = Shape<RT>;
    constexpr int NS = S::kStages, T = kTeams, KG = kSplit, KB = kBlocks / KG, kCols = S::kCols;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = base;
    float* slots = reinterpret_cast<float*>(ring + NS * kTileBytes);
    float2* slot_ml = reinterpret_cast<float2*>(slots + kConsumers * S::kSlotFloats);
    float* weights = reinterpret_cast<float*>(slot_ml + kConsumers * kCols);
    Plan& plan = *reinterpret_cast<Plan*>(weights + kConsumers * kCols * 8);
    uint64_t* bars = reinterpret_cast<uint64_t*>(&plan + 1);
    float* scales = reinterpret_cast<float*>(bars + 48);
    int* tickets = reinterpret_cast<int*>(scales + NS * 8);
    int* issued = tickets + kTickets;         // each stage's uses so far
    int* valid = issued + 16;                 // whether its tile has a page
    int* flags = valid + 16;                  // [0]: the CTA gives up; [1]: it has met V scales far apart
    Share& share_s = *reinterpret_cast<Share*>(flags + 4);
    const uint32_t full0 = ptx::smem_u32(bars), empty0 = full0 + 8 * 16, free0 = full0 + 8 * 32;
    const uint32_t filled = full0 + 8 * 40, joined = full0 + 8 * 41;
    volatile int* abort = flags;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        ptx::tma_prefetch_desc(&map_k);
        ptx::tma_prefetch_desc(&map_v);
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(full0 + 8 * s, 1);
            ptx::mbar_init(empty0 + 8 * s, KG);
        }
        for (int w = 0; w < kConsumers; ++w) ptx::mbar_init(free0 + 8 * w, 1);
        ptx::mbar_init(filled, kConsumers);
        ptx::mbar_init(joined, kConsumers);
        ptx::mbar_init_fence();
        flags[0] = flags[1] = 0;
        for (int s = 0; s < 16; ++s) issued[s] = 0;
    }
    for (int i = tid; i < kTickets; i += kAttnThreads) tickets[i] = 0;
    __syncthreads();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    int status = 0;
    const Share share = make_plan<kAttnThreads>(plan, a);
    if ((int)blockIdx.x >= share.n_ctas) return;
    if (tid == 0) share_s = share;

    if (warp >= kConsumers) {
        ptx::set_max_regs_dec<kProducerRegs>();
        // ------------------------------------------------------------ producers
        // Four warps take the tiles in turn (one alone issued a tile in 0.5 us, longer than a tile takes to arrive).
        // A lane looks up a tile's page, 32 at once; then the warp issues them one by one, a copy a lane.
        const int n = share.n, pw = warp - kConsumers;
        int last = -1;
        bool given_up = false;
        for (int i0 = pw; i0 < n && !given_up; i0 += 4 * 32) {
            int row = -1;
            if (i0 + 4 * lane < n) row = tile_row(plan, a, share.c0 + i0 + 4 * lane, status);
            for (int l = 0; l < 32 && i0 + 4 * l < n; ++l) {
                const int i = i0 + 4 * l, s = i % NS, use = i / NS, r = __shfl_sync(0xffffffffu, row, l);
                if (use > 0 && !page_wait(issued + s, use - 1, empty0 + 8 * s, (use - 1) & 1, abort, status)) {
                    given_up = true;
                    break;
                }
                const uint32_t bar = full0 + 8 * s, dst = ptx::smem_u32(ring + s * kTileBytes);
                if (lane == 0) {
                    valid[s] = r >= 0;
                    if (r >= 0) ptx::mbar_arrive_expect_tx(bar, kTileBytes + 32);
                    else ptx::mbar_arrive(bar);
                    // (no fence: what the reader must not miss, the end of the stage's last use, came before this
                    // lane's wait for the stage, and shared memory has one order)
                    *(volatile int*)(issued + s) = use + 1;
                }
                __syncwarp();
                if (r >= 0) {
                    if (lane < 2)
                        ptx::tma_load_2d(dst + lane * kHeadBytes, lane ? &map_v : &map_k, 0, r * kPage, bar);
                    else if (lane < 4)
                        ptx::bulk_load(ptx::smem_u32(scales + 8 * s) + 16 * (lane - 2),
                                       (lane == 2 ? a.k_scale : a.v_scale) + (size_t)r * kBlocks, 16, bar);
                }
                last = i;
            }
        }
        // no CTA ends with copies under way, even if its consumers gave up
        for (; last >= 0 && last > n - 1 - NS; last -= 4)
            ptx::mbar_wait(full0 + 8 * (last % NS), (last / NS) & 1, nullptr, kWaitNs);
    } else {
        // ------------------------------------------------------------ consumers
        ptx::set_max_regs_inc<kConsumerRegs>();
        const int team = warp / KG, kg = warp % KG;
        const int g = lane >> 2, j = lane & 3;
        const int kperm = (g & ~1) ^ ((g & 1) ? 5 : 0);       // this lane's key row of each eight
        const int heads = a.n_kv * a.group, cols_used = a.n_rows * a.group;
        float* slot = slots + (size_t)warp * S::kSlotFloats;
        float2* my_ml = slot_ml + warp * kCols;
        // how often the slot has been filled for a single warp's join, and for a common one; which was the last
        int uses = 0, joins = 0, slot_use = 0;
        bool given_up = false, far = false;
        Walk walk(share);
        while (!given_up && walk.next(plan, a, share.n)) {
            const int b = walk.b, h = walk.h, len = walk.len, live = walk.live, i_begin = walk.begin, i_end = walk.end;
            const int seg = walk.seg, seg_len = i_end - i_begin;
            const bool whole = walk.whole;
            int i = i_begin + ((team - i_begin) & (T - 1));
            if (i >= i_end) continue;
            // Q, each row brought to f16's upper range by a power of two (exact but for elements below 2^-31 of the row's
            // largest, which lose digits to 2^-39 and are 0 from there); f turns accumulated scores into base-2 exponents
            uint32_t qf[RT][8][2];
            float f[RT][2], m[RT][2], l[RT][2];
            int p[RT][2];                                     // positions of the columns' rows
            float o[RT][8][4];
            {
                uint4 raw[RT][4];
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    const int c = 8 * n + g;
#pragma unroll
                    for (int e = 0; e < 4; ++e) raw[n][e] = make_uint4(0u, 0u, 0u, 0u);
                    if (c < cols_used && plan.col_row[c] < live) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            a.q + (((size_t)b * a.n_rows + plan.col_row[c]) * heads + h * a.group + plan.col_head[c]) * kD +
                            16 * j);
                        raw[n][0] = __ldg(src);
                        raw[n][1] = __ldg(src + 1);
                        raw[n][2] = __ldg(src + 8);
                        raw[n][3] = __ldg(src + 9);
                    }
                }
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[n]);
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int up = min(max(268 - (int)(top >> 7), 1), 253);
                    const float by = __uint_as_float((uint32_t)up << 23);
                    const float back = __uint_as_float((uint32_t)(254 - up) << 23) * a.scale_log2;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t v = w[2 * s + e];
                            qf[n][s][e] = pack_f16(__uint_as_float(v << 16) * by, __uint_as_float(v & 0xFFFF0000u) * by);
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f[n][e] = __shfl_sync(0xffffffffu, back, (2 * j + e) * 4);
                        m[n][e] = kNoScore;
                        l[n][e] = 0.0f;
                        p[n][e] = len - live + min((int)plan.col_row[8 * n + 2 * j + e], live - 1);
                    }
#pragma unroll
                    for (int d = 0; d < 8; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][d][e] = 0.0f;
                }
            }
            float R = 0.0f, inv_r = 0.0f, vmin = INFINITY;
            for (; i < i_end; i += T) {
                const int st = i % NS;
                if (!page_wait(issued + st, i / NS, full0 + 8 * st, (i / NS) & 1, abort, status)) {
                    given_up = true;
                    break;
                }
                if (valid[st]) {
                    const unsigned char* kt = ring + st * kTileBytes;
                    const unsigned char* vt = kt + kHeadBytes;
                    const float* sc = scales + 8 * st;
                    const int key0 = (walk.page0 + (i - i_begin)) * kPage;
                    // some row does not see all of the page's keys
                    const bool edge = key0 + kPage - 1 > len - live || (a.window > 0 && key0 < len - a.window);
                    // this warp's KB blocks; no row sees those past the sequence, where scales may be anything, and those
                    // before its first window
                    const int k0 = kg * KB;
                    const bool none = edge && (key0 + k0 * kBlock >= len ||
                                               key0 + (k0 + KB) * kBlock <= seen_from(len, live, a.window));
                    if (!none) {
                        float vs[KB];
                        float vmax = 0.0f;
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            vs[k] = sc[kBlocks + k0 + k];
                            if (edge) {
                                const int at = key0 + (k0 + k) * kBlock;
                                if (at >= len || at + kBlock <= seen_from(len, live, a.window)) vs[k] = 0.0f;
                            }
                            vmax = fmaxf(vmax, vs[k]);
                            vmin = fminf(vmin, vs[k] > 0.0f ? vs[k] : INFINITY);
                        }
                        if (vmax > R) {
                            const uint32_t next = (__float_as_uint(vmax) + 0x7FFFFFu) & 0x7F800000u;
                            const float up = __uint_as_float(min(next, 0x7F000000u));
                            const float by = R / up;
                            R = up;
                            inv_r = 1.0f / up;
#pragma unroll
                            for (int n = 0; n < RT; ++n)
#pragma unroll
                                for (int d = 0; d < 8; ++d)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[n][d][e] *= by;
                        }
                        // scores of 16 KB keys
                        float s[KB][RT][4];
#pragma unroll
                        for (int k = 0; k < KB; ++k)
#pragma unroll
                            for (int n = 0; n < RT; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[k][n][e] = 0.0f;
                        const unsigned char* row = kt + (k0 * kBlock + kperm) * kD;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int at = ((j + 4 * u) ^ kperm) * 16;
                            uint4 ra[KB], rb[KB];
#pragma unroll
                            for (int k = 0; k < KB; ++k) {
                                ra[k] = *reinterpret_cast<const uint4*>(row + k * kBlock * kD + at);
                                rb[k] = *reinterpret_cast<const uint4*>(row + (k * kBlock + 8) * kD + at);
                            }
#pragma unroll
                            for (int w = 0; w < 4; ++w)
#pragma unroll
                                for (int k = 0; k < KB; ++k) {
                                    const uint32_t wa[4] = {ra[k].x, ra[k].y, ra[k].z, ra[k].w};
                                    const uint32_t wb[4] = {rb[k].x, rb[k].y, rb[k].z, rb[k].w};
                                    uint32_t a0, a1, a2, a3;
                                    widen<kInt8>(wa[w], a0, a2);
                                    widen<kInt8>(wb[w], a1, a3);
#pragma unroll
                                    for (int n = 0; n < RT; ++n)
                                        mma_f16(s[k][n], a0, a1, a2, a3, qf[n][4 * u + w][0], qf[n][4 * u + w][1]);
                                }
                        }
                        // exponents y = t - m + kShift and masks; a column without a score yet counts from 0 and
                        // gets its reference now, another one when a score has passed the old one by kLazy
                        bool raise = false;
                        float top[RT][2];
#pragma unroll
                        for (int n = 0; n < RT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float z = kShift - (m[n][e] == kNoScore ? 0.0f : m[n][e]);
                                top[n][e] = -INFINITY;
#pragma unroll
                                for (int k = 0; k < KB; ++k) {
                                    const float fk = f[n][e] * sc[k0 + k];
                                    float x0 = fmaf(s[k][n][e], fk, z), x1 = fmaf(s[k][n][2 + e], fk, z);
                                    if (edge) {
                                        const int key = key0 + (k0 + k) * kBlock + kperm;
                                        const int lo = a.window > 0 ? p[n][e] - a.window : -1;
                                        if (key > p[n][e] || key <= lo) x0 = -INFINITY;
                                        if (key + 8 > p[n][e] || key + 8 <= lo) x1 = -INFINITY;
                                    }
                                    s[k][n][e] = x0;
                                    s[k][n][2 + e] = x1;
                                    top[n][e] = fmaxf(top[n][e], fmaxf(x0, x1));
                                }
                                raise = raise || top[n][e] > (m[n][e] == kNoScore ? -INFINITY : kShift + kLazy);
                            }
                        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                            for (int n = 0; n < RT; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float now = top[n][e];
                                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 4));
                                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
                                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
                                    const bool none_yet = m[n][e] == kNoScore;
                                    float up = 0.0f;
                                    if (now > -INFINITY) up = none_yet ? now - kShift : fmaxf(now - kShift, 0.0f);
                                    if (now > -INFINITY) m[n][e] = (none_yet ? 0.0f : m[n][e]) + up;
                                    const float by = none_yet ? 1.0f : ptx::ex2(-up);      // (sums of nothing are 0)
                                    l[n][e] *= by;
#pragma unroll
                                    for (int k = 0; k < KB; ++k) {
                                        s[k][n][e] -= up;
                                        s[k][n][2 + e] -= up;
                                    }
#pragma unroll
                                    for (int d = 0; d < 8; ++d) {
                                        o[n][d][e] *= by;
                                        o[n][d][2 + e] *= by;
                                    }
                                }
                        }
                        // weights
                        uint32_t pf[KB][RT][2];
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            const float r = vs[k] * inv_r;
#pragma unroll
                            for (int n = 0; n < RT; ++n) {
                                const float p0 = ptx::ex2(s[k][n][0]), p1 = ptx::ex2(s[k][n][1]);
                                const float p2 = ptx::ex2(s[k][n][2]), p3 = ptx::ex2(s[k][n][3]);
                                l[n][0] += p0 + p2;
                                l[n][1] += p1 + p3;
                                pf[k][n][0] = transpose8(pack_f16(p0 * r, p1 * r));
                                pf[k][n][1] = transpose8(pack_f16(p2 * r, p3 * r));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            const int even = 2 * j, odd = (2 * j) ^ 5;
                            const unsigned char* blk = vt + (k0 + k) * kBlock * kD;
                            uint4 w0 = *reinterpret_cast<const uint4*>(blk + even * kD + (g ^ even) * 16);
                            uint4 w1 = *reinterpret_cast<const uint4*>(blk + odd * kD + (g ^ odd) * 16);
                            uint4 w2 = *reinterpret_cast<const uint4*>(blk + (even + 8) * kD + (g ^ even) * 16);
                            uint4 w3 = *reinterpret_cast<const uint4*>(blk + (odd + 8) * kD + (g ^ odd) * 16);
                            if (!kInt8 && edge) {      // what lies past the sequence may be NaN
                                const int key = key0 + (k0 + k) * kBlock;
                                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                                if (key + even >= len) w0 = zero;
                                if (key + odd >= len) w1 = zero;
                                if (key + even + 8 >= len) w2 = zero;
                                if (key + odd + 8 >= len) w3 = zero;
                            }
                            const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
                            const uint32_t u2[4] = {w2.x, w2.y, w2.z, w2.w}, u3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                // dimensions 4 w, 4 w + 1 of the even and odd keys side by side, then 4 w + 2, 4 w + 3
                                uint32_t a0, a1, a2, a3;
                                widen<kInt8>(__byte_perm(u0[w], u1[w], 0x5140), a0, a1);
                                widen<kInt8>(__byte_perm(u2[w], u3[w], 0x5140), a2, a3);
#pragma unroll
                                for (int n = 0; n < RT; ++n)
                                    mma_f16(o[n][2 * w], a0, a1, a2, a3, pf[k][n][0], pf[k][n][1]);
                                widen<kInt8>(__byte_perm(u0[w], u1[w], 0x7362), a0, a1);
                                widen<kInt8>(__byte_perm(u2[w], u3[w], 0x7362), a2, a3);
#pragma unroll
                                for (int n = 0; n < RT; ++n)
                                    mma_f16(o[n][2 * w + 1], a0, a1, a2, a3, pf[k][n][0], pf[k][n][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty0 + 8 * st);
            }
            if (given_up) break;
            far = far || R > fminf(kFar * vmin, kHuge);
            // -------------------------------------------------------- sums of the segment, into the warp's slot
            const int active = min(T, seg_len) * KG;              // warps that have a part of it
            if (slot_use == 1 && !warp_wait(free0 + 8 * warp, (uses - 1) & 1, abort, status)) break;
            if (slot_use == 2 && !warp_wait(joined, (joins - 1) & 1, abort, status)) break;
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[n][e];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    const int c = 8 * n + 2 * j + e;
                    if (g == 0) my_ml[c] = make_float2(m[n][e] == kNoScore ? -INFINITY : m[n][e] - kShift, sum);
                    // dimensions 16 g .. 16 g + 15 of pair c: the lane's eight accumulator pairs in order
                    float4* dst = reinterpret_cast<float4*>(slot + c * kD);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        dst[4 * g + (w ^ j)] = make_float4(o[n][2 * w][e] * R, o[n][2 * w][2 + e] * R, o[n][2 * w + 1][e] * R,
                                                           o[n][2 * w + 1][2 + e] * R);
                }
            // the active warps, in the order of their tiles
            auto warp_of = [&](int t) { return (((i_begin & (T - 1)) + t / KG) & (T - 1)) * KG + t % KG; };
            // Pair c: the sum over the active warps, to the output if the segment is the whole head, else to this CTA's
            // part of it.
            auto join = [&](int c) {
                const int chunk = (lane & ~3) | ((lane & 3) ^ ((c >> 1) & 3)), t_mine = lane & 7;
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (t_mine < active) ml = slot_ml[warp_of(t_mine) * kCols + c];
                float4 v[8];
#pragma unroll
                for (int t = 0; t < T * KG; ++t)
                    if (t < active)
                        v[t] = reinterpret_cast<const float4*>(slots + (size_t)warp_of(t) * S::kSlotFloats + c * kD)[chunk];
                float top = ml.x;
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                float one = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.0f) : exp2f(ml.x - top);
                float sum = one * ml.y;
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                const size_t part = (size_t)(2 * blockIdx.x + (i_begin == 0 ? 0 : 1)) * kMaxCols + c;
                const int head = h * a.group + plan.col_head[c];
                const size_t row = ((size_t)b * a.n_rows + plan.col_row[c]) * heads + head;
                if (whole) {
                    const Finish fin = finish(top, sum, a.sink, head);
                    one *= fin.by;
                    if (lane == 0 && a.out_lse) a.out_lse[row] = fin.lse;
                } else if (lane == 0) {
                    a.part_ml[part] = make_float2(top, sum);
                }
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int t = 0; t < T * KG; ++t)
                    if (t < active) {
                        const float w = __shfl_sync(0xffffffffu, one, t);
                        acc.x += w * v[t].x;
                        acc.y += w * v[t].y;
                        acc.z += w * v[t].z;
                        acc.w += w * v[t].w;
                    }
                if (whole) store_row(a.out + row * kD + 4 * lane, acc);
                else reinterpret_cast<float4*>(a.part_o + part * kD)[lane] = acc;
            };
            // (rolled loops: this runs a few times in a CTA, from a cold instruction cache)
            if (seg_len >= T) {
                // every warp has a part: they meet, and share the columns
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(filled);
                if (!warp_wait(filled, joins & 1, abort, status)) break;
#pragma unroll 1
                for (int c = warp; c < live * a.group; c += kConsumers) join(c);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(joined);
                ++joins;
                slot_use = 2;
            } else {
                // the last of the active warps joins their columns; the others go on
                int last = 1;
                __threadfence_block();
                __syncwarp();
                if (lane == 0) {
                    int* ticket = tickets + (seg & (kTickets - 1));
                    last = atomicAdd(ticket, 1) == active - 1;
                    if (last) *ticket = 0;
                }
                last = __shfl_sync(0xffffffffu, last, 0);
                ++uses;
                slot_use = 1;
                if (!last) continue;
                __threadfence_block();
                __syncwarp();
                // weights first: eight lanes a column, one for each active warp; then the columns' rows
                float* by = weights + warp * kCols * 8;
                const size_t part = (size_t)(2 * blockIdx.x + (i_begin == 0 ? 0 : 1)) * kMaxCols;
                const int n_here = live * a.group;
#pragma unroll 1
                for (int c = lane >> 3; c < kCols; c += 4) {
                    const int t = lane & 7;
                    float2 ml = make_float2(-INFINITY, 0.0f);
                    if (t < active) ml = slot_ml[warp_of(t) * kCols + c];
                    float top = ml.x;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    float one = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.0f) : exp2f(ml.x - top);
                    float sum = one * ml.y;
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    if (c < n_here) {
                        if (whole) {
                            const int head = h * a.group + plan.col_head[c];
                            const Finish fin = finish(top, sum, a.sink, head);
                            one *= fin.by;
                            if (t == 0 && a.out_lse)
                                a.out_lse[((size_t)b * a.n_rows + plan.col_row[c]) * heads + head] = fin.lse;
                        } else if (t == 0) {
                            a.part_ml[part + c] = make_float2(top, sum);
                        }
                    }
                    by[c * 8 + t] = one;
                }
                __syncwarp();
#pragma unroll 2
                for (int c = 0; c < n_here; ++c) {
                    const int chunk = (lane & ~3) | ((lane & 3) ^ ((c >> 1) & 3));
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int t = 0; t < active; ++t) {
                        const float one = by[c * 8 + t];
                        const float* of = slots + (size_t)warp_of(t) * S::kSlotFloats;
                        const float4 v = reinterpret_cast<const float4*>(of + c * kD)[chunk];
                        acc.x += one * v.x;
                        acc.y += one * v.y;
                        acc.z += one * v.z;
                        acc.w += one * v.w;
                    }
                    const size_t out_row = ((size_t)b * a.n_rows + plan.col_row[c]) * heads + h * a.group + plan.col_head[c];
                    if (whole)
                        store_row(a.out + out_row * kD + 4 * lane, acc);
                    else
                        reinterpret_cast<float4*>(a.part_o + (part + c) * kD)[lane] = acc;
                }
                __syncwarp();
                if (lane < active) ptx::mbar_arrive(free0 + 8 * warp_of(lane));
            }
        }
        // -------------------------------------------------------- segments whose V scales lie far apart, again
        if (far && lane == 0) flags[1] = 1;
        static_assert(kConsumers == kExactWarps, "the consumers compute them");
        ptx::named_bar_sync(1, 32 * kConsumers);
        if (__builtin_expect(flags[1] != 0, 0)) {
            const Share again = share_s;
            exact_segments<kInt8>(a, plan, again, *reinterpret_cast<ExactSmem*>(slots));
        }
    }
    if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// RT: the 8-pair tiles that cover the call's pairs.
template <bool kInt8, int RT>
cudaError_t launch_shape(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    const cudaError_t e = ensure_smem_attr((const void*)attn_paged_kernel<kInt8, RT>, Shape<RT>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    pdl_config(&cfg, attr, dim3((unsigned)a.n_ctas), dim3(kAttnThreads), Shape<RT>::kBytes, stream);
    return cudaLaunchKernelEx(&cfg, attn_paged_kernel<kInt8, RT>, a, k, v);
}

// By the (row, query head) pairs of a KV head: up to 16 here, more on tcgen05 (paged_attn_tc.cuh).  Here and there, E4M3,
// us: 16 pairs of one 192K sequence 24.3 and 31.0, of 64 ragged sequences of 1 to 16K (8 heads) 96.5 and 117, of 64 of 0.1
// to 1.1K (2 heads) 23.6 and 25.9, of 32 in windows of 4,096 28.2 and 37.3, of 4 of 1K 14.6 and 14.1; 6 pairs of the same
// 21.0 and 30.7, 60.7 and 115, 16.2 and 24.0, 24.2 and 36.7, 11.1 and 13.5.  From 17 on this kernel needs a second warp a
// code or a third column tile: 48 pairs of one 192K sequence took 48 us here and 36.5 us there, 30 of 32 sequences in a
// window of 4,096 44 us and 35.6 us.
template <bool kInt8>
cudaError_t launch_format(const AttnPagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    const int cols = a.n_rows * a.group;
    if (cols <= 8) return launch_shape<kInt8, 1>(a, k, v, stream);
    if (cols <= kFewPairs) return launch_shape<kInt8, 2>(a, k, v, stream);
    if (cols <= 32) return tcg::launch<kInt8, 32>(a, stream);
    if (cols <= 48) return tcg::launch<kInt8, 48>(a, stream);
    return tcg::launch<kInt8, 64>(a, stream);
}

}  // namespace paged
}  // namespace va
