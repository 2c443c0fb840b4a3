// Operations on the pages of the cache (include/kv_pages.h): room for new tokens with copy on write, forking,
// freeing and reordering of sequences, copying and compaction.
//
// The reference counts are the allocator's whole state: a page without references is free and the
// lowest-numbered free page goes first, so no free list has to be kept in step and the outcome does not depend
// on the order in which threads run.  The plans (who gets which page) are integers: one CTA makes each, the
// copies that it asks for run in a launch of their own over all SMs, behind a programmatic dependency.
// Measured, graph-replayed: kv_page_compact of 1,500 live pages of 4,096 (2 heads, 4 layers: 250 MB) 56 us, of which the
// copy 38 us, 6.5 TB/s; kv_page_reorder and kv_page_extend behind three copies of the state, 32 x 8 hypotheses (4 layers, 2
// heads) 22 to 24 us, 1 x 4 (2 layers) 12 to 13 us.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace va {
namespace paged {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kScan = 16;                 // reference counts per thread and round of a plan's scan
constexpr int kMaxSeqs = VA_PAGED_MAX_SEQS;

// Workspace: the number of copies, then per page the copies' sources and destinations, the count of its
// holders, its first holder, and a list of free pages.
struct Workspace {
    int32_t *n_pairs, *src, *dst, *holders, *first, *list;
};
constexpr size_t kHeaderBytes = 256;
inline size_t page_words(int n_pages) { return ((size_t)n_pages + 63) / 64 * 64; }
inline Workspace split_workspace(void* base, int n_pages) {
    Workspace w;
    const size_t n = page_words(n_pages);
    w.n_pairs = static_cast<int32_t*>(base);
    w.src = w.n_pairs + kHeaderBytes / 4;
    w.dst = w.src + n;
    w.holders = w.dst + n;
    w.first = w.holders + n;
    w.list = w.first + n;
    return w;
}

// Inclusive scan of one int per thread over the CTA; `sums` holds kPlanWarps + 1 ints.  Every thread gets the
// scan up to itself; sums[kPlanWarps] is the total.
__device__ __forceinline__ int block_scan(int v, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int s = lane < kPlanWarps ? sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        sums[lane] = s;
    }
    __syncthreads();
    const int before = warp > 0 ? sums[warp - 1] : 0;
    if (threadIdx.x == 0) sums[kPlanWarps] = sums[kPlanWarps - 1];
    __syncthreads();
    return before + v;
}

// ----------------------------------------------------------------------------- extend
struct ExtendArgs {
    int32_t *table, *lens, *refs;
    const int32_t* n_new;
    int32_t* dev_status;
    int n_seqs, max_pages, n_pages;
    Workspace w;
};

struct PlanSmem {
    int x0[kMaxSeqs], upto[kMaxSeqs];                // a sequence's first entry; entries of the sequences up to it
    int sums[kPlanWarps + 1];
    int counts[kScan * kPlanWarps];
    int status, pairs, found;
    alignas(16) int page[kPlanThreads];              // of at most as many entries as threads: the shared pages, -2 = none,
    int list[kPlanThreads];                          // and the free pages to be handed out
};

// The free pages among kScan * kPlanThreads from c0 on (r: their counts, page c0 + i * kPlanThreads + tid in r[i]), in order
// behind the sm.found before, to the first `total` places of `list`.
__device__ __forceinline__ void list_free(const int (&r)[kScan], int c0, int total, PlanSmem& sm, int32_t* list) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned mask[kScan];
#pragma unroll
    for (int i = 0; i < kScan; ++i) mask[i] = __ballot_sync(0xffffffffu, r[i] == 0);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kScan; ++i) sm.counts[i * kPlanWarps + warp] = __popc(mask[i]);
    }
    __syncthreads();
    const int c = tid < kScan * kPlanWarps ? sm.counts[tid] : 0;
    const int s = block_scan(c, sm.sums);
    const int found = sm.found;
    if (tid < kScan * kPlanWarps) sm.counts[tid] = found + s - c;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
        if ((mask[i] >> lane) & 1u) {
            const int rank = sm.counts[i * kPlanWarps + warp] + __popc(mask[i] & ((1u << lane) - 1u));
            if (rank < total) list[rank] = c0 + i * kPlanThreads + tid;
        }
    }
    if (tid == 0) sm.found = found + sm.sums[kPlanWarps];
    __syncthreads();
}

// The table entries of all pages that will be written, numbered in order of (slot, entry).  Pages of one reference stay
// with their entry and need nothing; only for shared ones the holders are counted and the first one found.
//   Up to 1,024 entries (a decode step's are one or two a slot): a thread each, everything between the loads and the
//   stores in registers and shared memory, the first 16,384 counts loaded with the lengths: three round trips to memory.
//   More (prompts): in passes over the entries, with the holders and the free list in the workspace.
// kv_page_reorder and kv_page_extend of 1 x 4 and 32 x 8 hypotheses took 13.4 and 22.0 us with the passes alone (three
// copies of the state among them), 11.9 and 21.7 us so.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const ExtendArgs a) {
    __shared__ PlanSmem sm;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x;
    if (tid == 0) sm.status = sm.pairs = sm.found = 0;
    int counts[kScan];
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
        const int p = i * kPlanThreads + tid;
        counts[i] = p < a.n_pages ? a.refs[p] : 1;
    }
    int status = 0, len = 0, add = 0, mine = 0;
    if (tid < a.n_seqs) {
        len = a.lens[tid];
        add = a.n_new[tid];
        const long long end = (long long)len + add;
        if (len < 0 || add < 0) status |= VA_DEV_BAD_COUNT;
        else if (end > (long long)a.max_pages * kPage) status |= VA_DEV_BEYOND_CACHE;
        if (!status && add > 0) mine = (int)((end + kPage - 1) / kPage) - len / kPage;
        sm.x0[tid] = len / kPage;
    }
    const int upto = block_scan(mine, sm.sums);
    if (tid < a.n_seqs) sm.upto[tid] = upto;
    const int entries = sm.sums[kPlanWarps];
    __syncthreads();
    // entry i: its slot (the first whose entries reach past i), place in the table and page
    auto slot_of = [&](int i) {
        int lo = 0, hi = a.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sm.upto[mid] > i) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    auto in_slot = [&](int i, int b) { return i - (b > 0 ? sm.upto[b - 1] : 0); };
    auto place = [&](int i, int b) { return b * a.max_pages + sm.x0[b] + in_slot(i, b); };
    auto refuse = [&](int why) {
        if (tid == 0) {
            *a.w.n_pairs = 0;
            if (a.dev_status) atomicOr(a.dev_status, why);
        }
    };
    if (entries <= kPlanThreads) {
        int b = 0, at = 0, p = -1, n_refs = 0;
        if (tid < entries) {
            b = slot_of(tid);
            at = place(tid, b);
            p = a.table[at];
            n_refs = p >= 0 && p < a.n_pages ? a.refs[p] : 0;
            if (p < -1 || p >= a.n_pages || (p >= 0 && n_refs < 1)) status |= VA_DEV_BAD_PAGE;
        }
        sm.page[tid] = n_refs > 1 ? p : -2;
        if (status) atomicOr(&sm.status, status);
        const bool some = __syncthreads_or(n_refs > 1);
        if (sm.status) return refuse(sm.status);
        // a shared page stays with its first holder here if no entry outside this call's names it
        bool fresh = tid < entries && p < 0;
        if (some && n_refs > 1) {
            int holders = 0, first = tid;
#pragma unroll 4
            for (int j = 0; j < entries; j += 4) {       // (-2 behind the entries)
                const int4 q = *reinterpret_cast<const int4*>(sm.page + j);
                const int here = (q.x == p) + (q.y == p) + (q.z == p) + (q.w == p);
                if (here && j < first) first = min(first, q.x == p ? j : q.y == p ? j + 1 : q.z == p ? j + 2 : j + 3);
                holders += here;
            }
            fresh = holders != n_refs || first != tid;
        }
        const int rank = block_scan(fresh ? 1 : 0, sm.sums) - 1, total = sm.sums[kPlanWarps];
        __syncthreads();
        if (total > 0) list_free(counts, 0, total, sm, sm.list);
        for (int c0 = kScan * kPlanThreads; c0 < a.n_pages && sm.found < total; c0 += kScan * kPlanThreads) {
#pragma unroll
            for (int i = 0; i < kScan; ++i) {
                const int q = c0 + i * kPlanThreads + tid;
                counts[i] = q < a.n_pages ? a.refs[q] : 1;
            }
            list_free(counts, c0, total, sm, sm.list);
        }
        if (sm.found < total) return refuse(VA_DEV_NO_PAGES);
        if (fresh) {
            const int page = sm.list[rank];
            a.table[at] = page;
            a.refs[page] = 1;
            if (p >= 0) {
                atomicSub(a.refs + p, 1);
                if (in_slot(tid, b) == 0 && a.lens[b] % kPage != 0) {      // only a slot's first entry can hold positions
                    const int j = atomicAdd(&sm.pairs, 1);
                    a.w.src[j] = p;
                    a.w.dst[j] = page;
                }
            }
        }
        __syncthreads();
        if (tid < a.n_seqs && add > 0) a.lens[tid] = len + add;
        if (tid == 0) *a.w.n_pairs = sm.pairs;
        return;
    }
    bool shared = false;
    for (int i = tid; i < entries; i += kPlanThreads) {
        const int p = a.table[place(i, slot_of(i))];
        const int r = p >= 0 && p < a.n_pages ? a.refs[p] : 0;
        if (p < -1 || p >= a.n_pages || (p >= 0 && r < 1)) {
            status |= VA_DEV_BAD_PAGE;
        } else if (r > 1) {
            shared = true;
            a.w.holders[p] = 0;
            a.w.first[p] = 0x7FFFFFFF;
        }
    }
    if (status) atomicOr(&sm.status, status);
    const bool some_shared = __syncthreads_or(shared);
    if (sm.status) return refuse(sm.status);
    if (some_shared) {
        for (int i = tid; i < entries; i += kPlanThreads) {
            const int p = a.table[place(i, slot_of(i))];
            if (p >= 0 && a.refs[p] > 1) {
                atomicAdd(a.w.holders + p, 1);
                atomicMin(a.w.first + p, i);
            }
        }
        __syncthreads();
        // first[p] stays the entry that keeps page p, or becomes -1: its first holder keeps it if no entry outside
        // this call's names it
        for (int i = tid; i < entries; i += kPlanThreads) {
            const int p = a.table[place(i, slot_of(i))];
            if (p >= 0 && a.refs[p] > 1 && __ldcg(a.w.first + p) == i && __ldcg(a.w.holders + p) != a.refs[p])
                __stcg(a.w.first + p, -1);
        }
        __syncthreads();
    }
    auto gets_new = [&](int i, int p) { return p < 0 || (a.refs[p] > 1 && __ldcg(a.w.first + p) != i); };
    int total = 0;
    for (int i0 = 0; i0 < entries; i0 += kPlanThreads) {
        const int i = i0 + tid;
        total += __syncthreads_count(i < entries && gets_new(i, a.table[place(i, slot_of(i))]));
    }
    // the `total` lowest-numbered free pages, in order
    if (total > 0) list_free(counts, 0, total, sm, a.w.list);
    for (int c0 = kScan * kPlanThreads; c0 < a.n_pages && sm.found < total; c0 += kScan * kPlanThreads) {
#pragma unroll
        for (int i = 0; i < kScan; ++i) {
            const int p = c0 + i * kPlanThreads + tid;
            counts[i] = p < a.n_pages ? a.refs[p] : 1;
        }
        list_free(counts, c0, total, sm, a.w.list);
    }
    if (sm.found < total) return refuse(VA_DEV_NO_PAGES);
    // Hand them out; the list keeps the shared page that each replaces, whose count changes once all have chosen.
    int rank0 = 0;
    for (int i0 = 0; i0 < entries; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int at = 0, b = 0, p = 0;
        bool fresh = false;
        if (i < entries) {
            b = slot_of(i);
            at = place(i, b);
            p = a.table[at];
            fresh = gets_new(i, p);
        }
        const int rank = rank0 + block_scan(fresh ? 1 : 0, sm.sums) - 1;
        rank0 += sm.sums[kPlanWarps];
        if (fresh) {
            const int page = a.w.list[rank];
            a.table[at] = page;
            a.refs[page] = 1;
            a.w.list[rank] = p;
            // only a slot's first entry can hold positions already
            if (p >= 0 && in_slot(i, b) == 0 && a.lens[b] % kPage != 0) {
                const int j = atomicAdd(&sm.pairs, 1);
                a.w.src[j] = p;
                a.w.dst[j] = page;
            }
        }
        __syncthreads();
    }
    for (int r = tid; r < total; r += kPlanThreads) {
        const int p = a.w.list[r];
        if (p >= 0) atomicSub(a.refs + p, 1);
    }
    __syncthreads();
    if (tid < a.n_seqs && add > 0) a.lens[tid] = len + add;
    if (tid == 0) *a.w.n_pairs = sm.pairs;
}

// ----------------------------------------------------------------------------- copies of pages
struct CopyArgs {
    const int32_t *src, *dst;
    const int32_t* n_pairs_dev;   // the number of copies, or null: n_pairs
    int n_pairs;
    uint4 *k_codes, *v_codes, *k_scale, *v_scale;
    int n_pages, n_layers, n_kv;
    int32_t* dev_status;
    // kv_page_compact: the table's entries follow
    int32_t* table;
    long long n_entries;
    const int32_t* moved_to;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = kHeadBytes / 16;   // 16-byte pieces of one page and head

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const CopyArgs a) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x;
    const int n = a.n_pairs_dev ? __ldcg(a.n_pairs_dev) : a.n_pairs;
    // one unit: one head's codes (8 KB) and scales (16 bytes) of K or V of one page in one layer (fewer than 2^26 of
    // 8 KB fit on a GPU)
    const unsigned units = (unsigned)n * a.n_layers * a.n_kv * 2u;
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
        const unsigned h = u % (unsigned)a.n_kv, rest = u / (unsigned)a.n_kv;
        const bool is_v = rest & 1u;
        const unsigned layer = (rest >> 1) % (unsigned)a.n_layers, i = (rest >> 1) / (unsigned)a.n_layers;
        const int from = __ldcg(a.src + i), to = __ldcg(a.dst + i);
        if (from < 0 || to < 0 || from >= a.n_pages || to >= a.n_pages) {
            if (tid == 0 && a.dev_status) atomicOr(a.dev_status, VA_DEV_BAD_PAGE);
            continue;
        }
        const size_t at_from = ((size_t)layer * a.n_pages + from) * a.n_kv + h;
        const size_t at_to = ((size_t)layer * a.n_pages + to) * a.n_kv + h;
        uint4* codes = is_v ? a.v_codes : a.k_codes;
        uint4* scale = is_v ? a.v_scale : a.k_scale;
        uint4 x[kCopyVecs / kCopyThreads];
#pragma unroll
        for (int c = 0; c < kCopyVecs / kCopyThreads; ++c) x[c] = __ldcs(codes + at_from * kCopyVecs + c * kCopyThreads + tid);
        if (tid == 0) scale[at_to] = scale[at_from];
#pragma unroll
        for (int c = 0; c < kCopyVecs / kCopyThreads; ++c) codes[at_to * kCopyVecs + c * kCopyThreads + tid] = x[c];
    }
    if (a.table) {
        for (long long e = (long long)blockIdx.x * kCopyThreads + tid; e < a.n_entries;
             e += (long long)gridDim.x * kCopyThreads) {
            const int p = a.table[e];
            if (p == -1) continue;
            const int to = p >= 0 && p < a.n_pages ? __ldcg(a.moved_to + p) : -1;
            if (to < 0 && a.dev_status) atomicOr(a.dev_status, VA_DEV_BAD_PAGE);
            if (to != p) a.table[e] = to;
        }
    }
}

static cudaError_t launch_copy(const CopyArgs& a, long long most_units, cudaStream_t stream) {
    // eight CTAs an SM keep 64 KB of loads in flight on each
    const int sms = device_sm_count();
    const long long most = 8ll * (sms > 0 ? sms : 148);
    long long work = most_units;
    const auto entry_work = (a.n_entries + kCopyThreads - 1) / kCopyThreads;
    if (a.table && work < entry_work) work = entry_work;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    pdl_config(&cfg, attr, dim3((unsigned)(work < 1 ? 1 : (work > most ? most : work))), dim3(kCopyThreads), 0, stream);
    return cudaLaunchKernelEx(&cfg, page_copy_kernel, a);
}

// ----------------------------------------------------------------------------- compaction
struct CompactArgs {
    int32_t *refs, *moved_to, *n_live;
    int n_pages;
    Workspace w;
};

// The live pages from n on (n live pages in all) are paired with the free ones below n, both in order.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
    __shared__ PlanSmem sm;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int live = 0;
    for (int p = tid; p < a.n_pages; p += kPlanThreads) live += a.refs[p] > 0;
    block_scan(live, sm.sums);
    const int n = sm.sums[kPlanWarps];
    __syncthreads();
    // below n the free pages are listed (destinations), from n on the live ones (sources): one rank each
    int below = 0, above = 0;
    for (int c0 = 0; c0 < a.n_pages; c0 += kScan * kPlanThreads) {
        unsigned mask[kScan];
        bool is_live[kScan];
#pragma unroll
        for (int i = 0; i < kScan; ++i) {
            const int p = c0 + i * kPlanThreads + tid;
            is_live[i] = p < a.n_pages && a.refs[p] > 0;
            const bool listed = p < a.n_pages && (p < n ? !is_live[i] : is_live[i]);
            mask[i] = __ballot_sync(0xffffffffu, listed);
        }
        // two scans, of the pages below n and of the others
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (lane < kScan) {
                const int p0 = c0 + lane * kPlanThreads + warp * 32;    // this warp's 32 pages of round `lane`
                unsigned m = 0;
#pragma unroll
                for (int i = 0; i < kScan; ++i) m = lane == i ? mask[i] : m;
                const int inside = min(max(n - p0, 0), 32);             // how many of them lie below n
                const unsigned lower = inside >= 32 ? 0xffffffffu : (1u << inside) - 1u;
                sm.counts[lane * kPlanWarps + warp] = __popc(m & (side == 0 ? lower : ~lower));
            }
            __syncthreads();
            const int c = tid < kScan * kPlanWarps ? sm.counts[tid] : 0;
            const int s = block_scan(c, sm.sums);
            const int before = side == 0 ? below : above;
            if (tid < kScan * kPlanWarps) sm.counts[tid] = before + s - c;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kScan; ++i) {
                const int p = c0 + i * kPlanThreads + tid;
                if (((mask[i] >> lane) & 1u) && (p < n) == (side == 0)) {
                    const int p0 = p - lane;
                    const int inside = min(max(n - p0, 0), 32);
                    const unsigned lower = inside >= 32 ? 0xffffffffu : (1u << inside) - 1u;
                    const unsigned same = mask[i] & (side == 0 ? lower : ~lower);
                    const int rank = sm.counts[i * kPlanWarps + warp] + __popc(same & ((1u << lane) - 1u));
                    (side == 0 ? a.w.dst : a.w.src)[rank] = p;
                }
            }
            if (side == 0) below += sm.sums[kPlanWarps];
            else above += sm.sums[kPlanWarps];
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kScan; ++i) {
            const int p = c0 + i * kPlanThreads + tid;
            if (p < a.n_pages) a.moved_to[p] = is_live[i] ? p : -1;
        }
    }
    __syncthreads();
    // as many free pages lie below n as live ones from n on
    for (int i = tid; i < above; i += kPlanThreads) {
        const int from = a.w.src[i], to = a.w.dst[i];
        a.moved_to[from] = to;
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
    if (tid == 0) {
        *a.n_live = n;
        *a.w.n_pairs = above;
    }
}

// ----------------------------------------------------------------------------- reorder
struct ReorderArgs {
    int32_t *table, *lens, *refs;
    const int32_t* src;
    int32_t* dev_status;
    int n_seqs, max_pages, group, n_pages;
};

constexpr int kReorderThreads = 256;

// A CTA takes all slots' entries of kCols columns (one 32-byte sector a row): columns do not depend on one another, so
// the table is rewritten in place.  The counts are sums of +1 and -1, whatever the order.
constexpr int kCols = 8;
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const ReorderArgs a) {
    __shared__ int old[kMaxSeqs * kCols];
    __shared__ int from[kMaxSeqs];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, x0 = blockIdx.x * kCols;
    int status = 0;
    for (int j = tid; j < a.n_seqs; j += kReorderThreads) {
        const int s = a.src[j];
        const bool ok = s >= -1 && s < a.group;
        if (!ok) status |= VA_DEV_BAD_COUNT;
        from[j] = !ok ? j : (s < 0 ? -1 : j / a.group * a.group + s);
    }
#pragma unroll 8
    for (int c = tid; c < a.n_seqs * kCols; c += kReorderThreads) {
        const int j = c / kCols, x = x0 + c % kCols;
        old[c] = x < a.max_pages ? a.table[(size_t)j * a.max_pages + x] : -1;
    }
    __syncthreads();
    for (int c = tid; c < a.n_seqs * kCols; c += kReorderThreads) {
        const int j = c / kCols, x = x0 + c % kCols;
        const int was = old[c], now = from[j] < 0 ? -1 : old[from[j] * kCols + c % kCols];
        if (x >= a.max_pages || was == now) continue;
        a.table[(size_t)j * a.max_pages + x] = now;
        if (was != -1) {
            if (was >= 0 && was < a.n_pages) atomicSub(a.refs + was, 1);
            else status |= VA_DEV_BAD_PAGE;
        }
        if (now != -1) {
            if (now >= 0 && now < a.n_pages) atomicAdd(a.refs + now, 1);
            else status |= VA_DEV_BAD_PAGE;
        }
    }
    if (blockIdx.x == 0) {
        __syncthreads();
        for (int j = tid; j < a.n_seqs; j += kReorderThreads) old[j] = a.lens[j];
        __syncthreads();
        for (int j = tid; j < a.n_seqs; j += kReorderThreads) a.lens[j] = from[j] < 0 ? 0 : old[from[j]];
    }
    if (status && a.dev_status) atomicOr(a.dev_status, status);
}

static bool table_ok(const int32_t* table, int n_seqs, int max_pages) {
    return table && n_seqs >= 1 && n_seqs <= VA_PAGED_MAX_SEQS && max_pages >= 1 && max_pages <= 0x7FFFFFFF / kPage;
}

static CopyArgs copy_args(int n_pages, int n_layers, int n_kv, void* k_codes, void* v_codes, float* k_scale,
                          float* v_scale, int32_t* dev_status) {
    CopyArgs c = {};
    c.k_codes = static_cast<uint4*>(k_codes);
    c.v_codes = static_cast<uint4*>(v_codes);
    c.k_scale = reinterpret_cast<uint4*>(k_scale);
    c.v_scale = reinterpret_cast<uint4*>(v_scale);
    c.n_pages = n_pages;
    c.n_layers = n_layers;
    c.n_kv = n_kv;
    c.dev_status = dev_status;
    return c;
}

}  // namespace paged
}  // namespace va

extern "C" {

size_t va_page_ops_workspace_bytes(int n_seqs, int max_pages, int n_pages) {
    if (n_seqs < 1 || n_seqs > VA_PAGED_MAX_SEQS || max_pages < 1 || n_pages < 1) return 0;
    return va::paged::kHeaderBytes + 5 * sizeof(int32_t) * va::paged::page_words(n_pages);
}

va_status kv_page_extend(int32_t* table, int32_t* lens, const int32_t* n_new, int n_seqs, int max_pages, int32_t* refs,
                         int n_pages, int n_layers, int n_kv_heads, void* k_codes, void* v_codes, float* k_scale,
                         float* v_scale, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         va_stream stream) {
    using namespace va::paged;
    if (!table_ok(table, n_seqs, max_pages) || !lens || !n_new || !refs || !workspace || !aligned16(workspace))
        return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, n_layers, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    if ((long long)n_seqs * max_pages > 0x7FFFFFFFll) return VA_UNSUPPORTED;   // entries are numbered in 32 bits
    if (workspace_bytes < va_page_ops_workspace_bytes(n_seqs, max_pages, n_pages)) return VA_INVALID_ARG;
    ExtendArgs a;
    a.table = table; a.lens = lens; a.refs = refs; a.n_new = n_new; a.dev_status = dev_status;
    a.n_seqs = n_seqs; a.max_pages = max_pages; a.n_pages = n_pages;
    a.w = split_workspace(workspace, n_pages);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream);
    st = launched(cudaLaunchKernelEx(&cfg, extend_plan_kernel, a));
    if (st != VA_OK) return st;
    CopyArgs c = copy_args(n_pages, n_layers, n_kv_heads, k_codes, v_codes, k_scale, v_scale, dev_status);
    c.src = a.w.src;
    c.dst = a.w.dst;
    c.n_pairs_dev = a.w.n_pairs;
    return launched(launch_copy(c, 2ll * n_seqs * n_layers * n_kv_heads, (cudaStream_t)stream));
}

va_status kv_page_reorder(int32_t* table, int32_t* lens, int n_seqs, int max_pages, const int32_t* src, int group,
                          int32_t* refs, int n_pages, int32_t* dev_status, va_stream stream) {
    using namespace va::paged;
    if (!table_ok(table, n_seqs, max_pages) || !lens || !src || !refs || n_pages < 1) return VA_INVALID_ARG;
    if (group < 0 || group > n_seqs || (group > 0 && n_seqs % group != 0)) return VA_INVALID_ARG;
    ReorderArgs a;
    a.table = table; a.lens = lens; a.refs = refs; a.src = src; a.dev_status = dev_status;
    a.n_seqs = n_seqs; a.max_pages = max_pages; a.group = group > 0 ? group : n_seqs; a.n_pages = n_pages;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3((unsigned)((max_pages + kCols - 1) / kCols)), dim3(kReorderThreads), 0,
                   (cudaStream_t)stream);
    return launched(cudaLaunchKernelEx(&cfg, reorder_kernel, a));
}

va_status kv_page_copy(const int32_t* src, const int32_t* dst, int n_pairs, int n_pages, int n_layers, int n_kv_heads,
                       void* k_codes, void* v_codes, float* k_scale, float* v_scale, int32_t* dev_status,
                       va_stream stream) {
    using namespace va::paged;
    if (n_pairs < 0 || n_pairs > n_pages) return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, n_layers, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    if (n_pairs == 0) return VA_OK;
    if (!src || !dst) return VA_INVALID_ARG;
    CopyArgs c = copy_args(n_pages, n_layers, n_kv_heads, k_codes, v_codes, k_scale, v_scale, dev_status);
    c.src = src;
    c.dst = dst;
    c.n_pairs = n_pairs;
    return launched(launch_copy(c, 2ll * n_pairs * n_layers * n_kv_heads, (cudaStream_t)stream));
}

va_status kv_page_compact(int32_t* table, int n_seqs, int max_pages, int32_t* refs, int n_pages, int n_layers,
                          int n_kv_heads, void* k_codes, void* v_codes, float* k_scale, float* v_scale,
                          int32_t* moved_to, int32_t* n_live_pages, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, va_stream stream) {
    using namespace va::paged;
    if (!table_ok(table, n_seqs, max_pages) || !refs || !moved_to || !n_live_pages || !workspace || !aligned16(workspace))
        return VA_INVALID_ARG;
    va_status st = check_pool(k_codes, v_codes, k_scale, v_scale, n_layers, n_pages, n_kv_heads);
    if (st != VA_OK) return st;
    if (workspace_bytes < va_page_ops_workspace_bytes(n_seqs, max_pages, n_pages)) return VA_INVALID_ARG;
    CompactArgs a;
    a.refs = refs; a.moved_to = moved_to; a.n_live = n_live_pages; a.n_pages = n_pages;
    a.w = split_workspace(workspace, n_pages);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    va::pdl_config(&cfg, attr, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream);
    st = launched(cudaLaunchKernelEx(&cfg, compact_plan_kernel, a));
    if (st != VA_OK) return st;
    CopyArgs c = copy_args(n_pages, n_layers, n_kv_heads, k_codes, v_codes, k_scale, v_scale, dev_status);
    c.src = a.w.src;
    c.dst = a.w.dst;
    c.n_pairs_dev = a.w.n_pairs;
    c.table = table;
    c.n_entries = (long long)n_seqs * max_pages;
    c.moved_to = moved_to;
    return launched(launch_copy(c, (long long)n_pages * n_layers * n_kv_heads, (cudaStream_t)stream));
}

}  // extern "C"
