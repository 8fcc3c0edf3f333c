// Page operators of the paged KV cache: rows grow and shrink (rd_resize_pages),
// branch (rd_fork_pages), pages are copied (rd_copy_pages) and the pool compacted
// (rd_compact_pages).  Paged KV caching: NVIDIA blog "ReDrafter in TensorRT-LLM",
// introduction.
//
// Two kinds of kernel:
//  - table kernels: one cluster of eight CTAs does a whole step on the tables
//    (block table, pages held per row, references per page).  A page is free when
//    its reference count is zero; "the k-th lowest free page" is a rank over the
//    counts, so the outcome depends on the tables alone and never on the order
//    of atomics.  The work is a few hundred KB at most; what bounds it is the
//    chain of dependent L2 reads and cluster barriers, hence one cluster (a
//    hardware barrier instead of further launches) and no free list to keep.
//    Resizing 16 rows of 4,096 pages takes 7.2 us, 1,000 rows of 65,536 pages 14.7
//    (by clock reads, of 25,000 cycles: row demands 2,800, pages given back and the
//    barrier 7,100, reference counts 2,200, their ranks 2,300, then the new entries
//    9,900 in the first CTA against 900 in the others: the lowest free pages all lie in
//    its share); five forks with their 1.3 MB of data 13.
//  - the page copy: bulk copies (TMA) through a shared-memory ring, one issuing
//    thread per CTA, two CTAs per SM; a page of K or V is one contiguous block,
//    so nothing but the ring's depth and HBM bounds it.  300 pages of 131 KB in 8
//    layers (1.26 GB read and written) take 202 us with the launch that checks the
//    pairs: 6.2 TB/s, 0.92 of a plain copy (193 us, 6.5 TB/s, alone); compacting 1.0
//    GB 162 us, 200 forks of half pages in 6 layers (0.31 GB) 59 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "block_scan.cuh"
#include "rd_internal.cuh"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace {

// ------------------------------------------------------------- table kernels
constexpr int kTableCtas = 8;              // one cluster
constexpr int kTableThreads = kScanThreads;
constexpr int kTableWarps = kScanWarps;
static_assert(RD_MAX_PAGES == kTableCtas * kTableWarps * 32 * 32, "one 32-page word per lane");

struct ScanSmem {
    int warp_sum[kTableWarps];
    int cta_total[kTableCtas];             // written by every CTA of the cluster
    int boundary;                          // rd_compact_pages: live pages below n_live
};

// Exclusive scan of f(i), i < n, into out[0 .. n] (out[n] = the sum): thread t
// takes a contiguous share.
template <typename F>
__device__ __forceinline__ int cta_scan_array(int n, int* out, int* warp_sum, F&& f)
{
    const int per = (n + kTableThreads - 1) / kTableThreads;
    const int i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
        const int v = f(i);
        out[i] = v;
        sum += v;
    }
    int total;
    int run = cta_scan(sum, warp_sum, total);
    for (int i = i0; i < i1; ++i) {
        const int v = out[i];
        out[i] = run;
        run += v;
    }
    if (threadIdx.x == 0) out[n] = total;
    __syncthreads();
    return total;
}

// Pages of the whole pool over the cluster: warp w of the cluster owns the words
// (32 pages each) [w q, (w + 1) q); lane i < q holds word i's bits.
struct PageWords {
    int first;             // first page of this warp
    int q;                 // words of this warp
    uint32_t bits;         // lane i: bit k set iff page first + 32 i + k is free (refs == 0)
};

// words of a warp, for a pool of that many pages
__host__ __device__ __forceinline__ int words_per_warp(int num_pages)
{
    return ((num_pages + 31) / 32 + kTableCtas * kTableWarps - 1) / (kTableCtas * kTableWarps);
}

__device__ __forceinline__ PageWords read_free(const int32_t* refs, int num_pages, int rank)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PageWords p;
    p.q = words_per_warp(num_pages);
    p.first = (rank * kTableWarps + warp) * p.q * 32;
    p.bits = 0u;
#pragma unroll 4
    for (int i = 0; i < p.q; ++i) {
        const int page = p.first + 32 * i + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, page < num_pages && __ldcg(refs + page) == 0);
        if (lane == i) p.bits = m;
    }
    return p;
}

// Rank of this lane's first set bit over the cluster's words, and the cluster's
// total.  One cluster barrier; every CTA must have started (an earlier barrier).
__device__ __forceinline__ int cluster_rank(uint32_t bits, ScanSmem& sc, const cg::cluster_group& cl,
                                            int& total)
{
    const int rank = (int)cl.block_rank();
    int cta;
    const int before = cta_scan(__popc(bits), sc.warp_sum, cta);
    if (threadIdx.x < kTableCtas) *cl.map_shared_rank(&sc.cta_total[rank], threadIdx.x) = cta;
    cl.sync();
    int base = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kTableCtas; ++i) {
        if (i < rank) base += sc.cta_total[i];
        total += sc.cta_total[i];
    }
    return base + before;
}

// f(page, rank) for every set bit of rank < limit, one page per lane.
template <typename F>
__device__ __forceinline__ void for_ranked(const PageWords& p, uint32_t bits, int base, int limit, F&& f)
{
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < p.q; ++i) {
        const uint32_t m = __shfl_sync(0xffffffffu, bits, i);
        const int b = __shfl_sync(0xffffffffu, base, i);
        if (m == 0u || b >= limit) continue;
        const int r = b + __popc(m & ((1u << lane) - 1u));
        if (((m >> lane) & 1u) && r < limit) f(p.first + 32 * i + lane, r);
    }
}

// last i in [0, n) with off[i] <= k (off ascending, off[0] <= k)
__device__ __forceinline__ int last_at_most(const int* off, int n, int k)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Rows grow and shrink.  Every CTA scans the rows' demands for itself (a few KB);
// the rows' shrinking, the free ranks and the new entries are split over the
// cluster.
__global__ void __launch_bounds__(kTableThreads, 1)
resize_kernel(int32_t* block_table, int R, int max_pages, int32_t* row_pages, int32_t* refs,
              int num_pages, const int32_t* __restrict__ new_lens, int page_size, int32_t* status)
{
    extern __shared__ int dyn[];
    int* off = dyn;                        // [R + 1] new pages of the rows before
    int* have = dyn + R + 1;               // [R] pages held at the start, -1: invalid row
    int* want = have + R;                  // [R] pages after the call
    __shared__ ScanSmem sc;
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();

    const int demand = cta_scan_array(R, off, sc.warp_sum, [&](int r) {
        int h = __ldcg(row_pages + r);
        const int n = __ldg(new_lens + r);
        const int w = n < 0 ? h : n == 0 ? 0 : (n - 1) / page_size + 1;
        if (h < 0 || h > max_pages || w > max_pages) {
            if (rank == 0) rd_flag(status, RD_DEV_BAD_LENGTH);
            h = -1;
        }
        have[r] = h;
        want[r] = w;
        return h < 0 ? 0 : max(0, w - h);
    });
    // give pages back: as many lanes a row as leaves every row its own, four entries
    // of a lane on the way at once
    constexpr int kAll = kTableCtas * kTableThreads, kAtOnce = 4;
    const int lanes = R <= kAll / 32 ? 32 : R <= kAll / 16 ? 16 : 8;
    const int me = rank * kTableThreads + (int)threadIdx.x;
    for (int r = me / lanes; r < R; r += kAll / lanes) {
        const int h = have[r];
        if (h < 0) continue;
        int32_t* row = block_table + (size_t)r * max_pages;
        // (entries counted unsigned: the last step may end behind 2^31)
        const uint32_t end = (uint32_t)h, step = (uint32_t)lanes;
        for (uint32_t j0 = (uint32_t)want[r] + (uint32_t)(me % lanes); j0 < end; j0 += step * kAtOnce) {
            int page[kAtOnce], held[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) page[e] = j0 + e * step < end ? __ldcg(row + j0 + e * step) : -1;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e)
                held[e] = page[e] >= 0 && page[e] < num_pages ? atomicSub(refs + page[e], 1) : 0;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                if (j0 + e * step >= end) continue;
                row[j0 + e * step] = -1;
                if (held[e] <= 0) {
                    rd_flag(status, RD_DEV_BAD_INDEX);
                    // held by nobody: leave it free
                    if (page[e] >= 0 && page[e] < num_pages) atomicAdd(refs + page[e], 1);
                }
            }
        }
    }
    cl.sync();
    int n_free = 0;
    if (demand > 0) {
        const PageWords p = read_free(refs, num_pages, rank);
        const int base = cluster_rank(p.bits, sc, cl, n_free);
        for_ranked(p, p.bits, base, min(demand, n_free), [&](int page, int k) {
            const int r = last_at_most(off, R, k);
            if (off[r + 1] > n_free) return;                    // the row does not fit
            block_table[(size_t)r * max_pages + have[r] + k - off[r]] = page;
            refs[page] = 1;
        });
    }
    for (int r = rank * kTableThreads + (int)threadIdx.x; r < R; r += kTableCtas * kTableThreads) {
        const int h = have[r];
        if (h < 0) continue;
        const bool fits = off[r + 1] == off[r] || off[r + 1] <= n_free;
        if (!fits) rd_flag(status, RD_DEV_OVERFLOW);
        else row_pages[r] = want[r];
    }
}

// Rows branch: tables here, the last pages' data by the copy kernel behind it, or
// here too when it is little (`here.pool` not null): no second launch, no list between
// them, and no workspace.  Measured here against a copy launch (one layer, 128 and
// 256 KB a page; L2 cold): 0.25 MB 18.6 against 19.3 us, 0.5 MB 18.8 / 19.1, 1 MB 20.0 / 19.4,
// 2 MB 21.9 / 20.7, 4 MB 25.6 / 20.2; warm 15.3 / 16.2, 14.8 / 14.4, 16.0 / 15.4, 18.1 / 15.3,
// 20.4 / 15.6.  So time alone would end it at 0.5 MB; up to 2 MB it costs 1 to 3 us
// and spares the caller the workspace.
constexpr size_t kForkHereBytes = 2u << 20;
struct ForkCopy {
    uint4* pool[2];                        // K, V
    int layers;
    size_t layer_vecs, page_vecs, row_bytes;
};
__global__ void __launch_bounds__(kTableThreads, 1)
fork_kernel(int32_t* block_table, int R, int max_pages, int32_t* row_pages, int32_t* refs, int num_pages,
            int32_t* ctx_lens, const int32_t* __restrict__ parent, const int32_t* __restrict__ child, int n,
            int page_size, int32_t* src, int32_t* dst, int32_t* used, const ForkCopy here, int32_t* status)
{
    extern __shared__ int dyn[];
    int* off = dyn;                        // [n + 1] new pages of the pairs before
    int* len = dyn + n + 1;                // [n] the parent's length, -1: no pair
    int* owner = len + n;                  // [R] first pair that names the row as its child
    // the pool's free pages before the call, a bit each: a parent's row may name one of
    // them by mistake, and the same call hands them out
    uint32_t* free_word = reinterpret_cast<uint32_t*>(owner + R);
    __shared__ ScanSmem sc;
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const int tid = threadIdx.x;
    const int warp = rank * kTableWarps + (tid >> 5), lane = tid & 31;
    // the copy kernel may start now; it waits for this grid before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    for (int r = tid; r < R; r += kTableThreads) owner[r] = 0x7fffffff;
    __syncthreads();
    for (int i = tid; i < n; i += kTableThreads) {
        const int p = __ldg(parent + i), c = __ldg(child + i);
        if (p >= 0 && c >= 0 && c < R) atomicMin(owner + c, i);
    }
    __syncthreads();
    const int demand = cta_scan_array(n, off, sc.warp_sum, [&](int i) {
        const int p = __ldg(parent + i), c = __ldg(child + i);
        int l = -1;
        if (p >= 0) {
            unsigned bad = 0u;
            if (p >= R || c < 0 || c >= R || c == p || owner[c] != i || __ldcg(row_pages + c) != 0) {
                bad = RD_DEV_BAD_INDEX;
            } else {
                l = __ldcg(ctx_lens + p);
                const int h = __ldcg(row_pages + p);
                if (l < 0 || h > max_pages || (l > 0 && (l - 1) / page_size + 1 > h)) {
                    bad = RD_DEV_BAD_LENGTH;
                    l = -1;
                }
            }
            if (bad && rank == 0) rd_flag(status, bad);
        }
        len[i] = l;
        return l >= 0 && l % page_size != 0 ? 1 : 0;
    });
    if (rank == 0 && dst != nullptr)
        for (int i = tid; i < n; i += kTableThreads) dst[i] = -1;
    // every CTA has read the tables before any is changed
    cl.sync();
    int n_free;
    const PageWords p = read_free(refs, num_pages, rank);
    if (lane < p.q)
        for (int i = 0; i < kTableCtas; ++i) cl.map_shared_rank(free_word, i)[p.first / 32 + lane] = p.bits;
    const int base = cluster_rank(p.bits, sc, cl, n_free);      // (and its barrier: the words have arrived)
    auto held = [&](int page) {
        return page >= 0 && page < num_pages && !((free_word[page >> 5] >> (page & 31)) & 1u);
    };
    for_ranked(p, p.bits, base, min(demand, n_free), [&](int page, int k) {
        const int i = last_at_most(off, n, k);
        const int full = len[i] / page_size;
        const int from = __ldcg(block_table + (size_t)__ldg(parent + i) * max_pages + full);
        block_table[(size_t)__ldg(child + i) * max_pages + full] = page;
        refs[page] = 1;
        if (!held(from)) {
            rd_flag(status, RD_DEV_BAD_INDEX);                  // nothing to copy
            return;
        }
        if (dst == nullptr) return;
        src[i] = from;
        dst[i] = page;
        used[i] = len[i] % page_size;
    });
    for (int i = warp; i < n; i += kTableCtas * kTableWarps) {
        const int l = len[i];
        if (l < 0) continue;
        if (off[i + 1] > off[i] && off[i] >= n_free) {          // no page for its last positions
            if (lane == 0) rd_flag(status, RD_DEV_OVERFLOW);
            continue;
        }
        const int from = __ldg(parent + i), to = __ldg(child + i), full = l / page_size;
        for (uint32_t j = lane; j < (uint32_t)full; j += 32) {
            const int page = __ldcg(block_table + (size_t)from * max_pages + j);
            block_table[(size_t)to * max_pages + j] = page;
            if (!held(page)) rd_flag(status, RD_DEV_BAD_INDEX);
            else atomicAdd(refs + page, 1);
        }
        if (lane == 0) {
            row_pages[to] = full + (off[i + 1] - off[i]);
            ctx_lens[to] = l;
        }
    }
    if (here.pool[0] == nullptr) return;
    cl.sync();                             // every new entry is written
    // one block of a page (K or V, one layer) per group of warps
    const int blocks = n * 2 * here.layers;
    const int share = max(1, kTableCtas * kTableWarps / blocks);       // warps of a block
    for (int q = warp; q < blocks * share; q += kTableCtas * kTableWarps) {
        const int blk = q / share, i = blk / (2 * here.layers), kl = blk % (2 * here.layers);
        const int l = len[i];
        if (l < 0 || l % page_size == 0 || off[i] >= n_free) continue;
        const int full = l / page_size;
        const int from = __ldcg(block_table + (size_t)__ldg(parent + i) * max_pages + full);
        const int to = __ldcg(block_table + (size_t)__ldg(child + i) * max_pages + full);
        if (!held(from)) continue;
        uint4* base = here.pool[kl & 1] + (size_t)(kl >> 1) * here.layer_vecs;
        const uint4* s = base + (size_t)from * here.page_vecs;
        uint4* d = base + (size_t)to * here.page_vecs;
        const size_t vecs = min(here.page_vecs, ((size_t)(l % page_size) * here.row_bytes + 15) / 16);
        constexpr int kAtOnce = 4;
        const size_t step = (size_t)share * 32;
        for (size_t v = (size_t)(q % share) * 32 + lane; v < vecs; v += step * kAtOnce) {
            uint4 x[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e)
                if (v + e * step < vecs) x[e] = __ldcg(s + v + e * step);
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e)
                if (v + e * step < vecs) d[v + e * step] = x[e];
        }
    }
}

// Compaction's plan: n_live = pages with references; the k-th lowest free page
// below n_live takes the k-th lowest live page at or above it.
__global__ void __launch_bounds__(kTableThreads, 1)
compact_plan_kernel(int32_t* refs, int num_pages, int32_t* remap, int32_t* n_live_out, int32_t* n_moves,
                    int32_t* src, int32_t* dst)
{
    __shared__ ScanSmem sc;
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const PageWords p = read_free(refs, num_pages, rank);
    cl.sync();                             // every CTA has started
    int n_free;
    const int base = cluster_rank(p.bits, sc, cl, n_free);
    const int n_live = num_pages - n_free;
    // free pages below n_live = moves: the lane whose word holds page n_live knows
    const int at = n_live - (p.first + 32 * lane);
    if (lane < p.q && at >= 0 && at < 32) {
        const int holes = base + __popc(p.bits & ((1u << at) - 1u));
        for (int i = 0; i < kTableCtas; ++i) *cl.map_shared_rank(&sc.boundary, i) = holes;
    }
    cl.sync();
    const int moves = n_free > 0 && n_live < num_pages ? sc.boundary : 0;
    for (int i = 0; i < p.q; ++i) {
        const uint32_t m = __shfl_sync(0xffffffffu, p.bits, i);
        const int page = p.first + 32 * i + lane;
        const int fr = __shfl_sync(0xffffffffu, base, i) + __popc(m & ((1u << lane) - 1u));   // free pages before
        const bool is_free = (m >> lane) & 1u;
        if (page >= num_pages) {
            // past the pool
        } else if (page < n_live) {
            remap[page] = is_free ? -1 : page;
            if (is_free) dst[fr] = page;
        } else if (is_free) {
            remap[page] = -1;
        } else {
            src[(page - fr) - (n_live - moves)] = page;
        }
    }
    cl.sync();
    for (int k = rank * kTableThreads + tid; k < moves; k += kTableCtas * kTableThreads) {
        const int s = __ldcg(src + k), d = __ldcg(dst + k);
        remap[s] = d;
        refs[d] = refs[s];
        refs[s] = 0;
    }
    if (rank == 0 && tid == 0) {
        *n_live_out = n_live;
        *n_moves = moves;
    }
}

// ------------------------------------------------------------------ page copy
// Pairs that may be copied side by side: pair i stays when its pages are in
// range and different, no earlier pair has its destination, and no pair writes
// its source.  Every thread compares its pair with the list, staged through
// shared memory.
constexpr int kResolveThreads = 256;
__device__ __forceinline__ int2 pair_at(const int32_t* src, const int32_t* dst, int k, int n, int num_pages)
{
    int2 v = make_int2(-1, -1);            // copies nothing
    if (k < n) {
        v = make_int2(__ldg(src + k), __ldg(dst + k));
        if (v.x < 0 || v.x >= num_pages || v.y < 0 || v.y >= num_pages || v.x == v.y) v = make_int2(-1, -1);
    }
    return v;
}
// whether a pair that copies nothing is wrong
__device__ __forceinline__ bool pair_wrong(const int32_t* src, const int32_t* dst, int k, int num_pages)
{
    const int s = __ldg(src + k), d = __ldg(dst + k);
    return s >= num_pages || (s >= 0 && s != d);
}
__global__ void __launch_bounds__(kResolveThreads)
resolve_kernel(const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, int num_pages,
               int32_t* src_out, int32_t* dst_out, int32_t* status)
{
    __shared__ int2 tile[kResolveThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int i = blockIdx.x * kResolveThreads + threadIdx.x;
    int2 mine = pair_at(src, dst, i, n, num_pages);
    bool clash = false;
    for (int k0 = 0; k0 < n; k0 += kResolveThreads) {
        __syncthreads();
        tile[threadIdx.x] = pair_at(src, dst, k0 + threadIdx.x, n, num_pages);
        __syncthreads();
        const int m = min(kResolveThreads, n - k0);
#pragma unroll 8
        for (int k = 0; k < m; ++k) {
            const int d = tile[k].y;       // (a pair of no effect has d = -1, and so have its x and y)
            clash |= (d == mine.x) | ((d == mine.y) & (k0 + k < i));
        }
    }
    if (i >= n) return;
    if (mine.y < 0) {
        if (pair_wrong(src, dst, i, num_pages)) rd_flag(status, RD_DEV_BAD_INDEX);
    } else if (clash) {
        rd_flag(status, RD_DEV_BAD_INDEX);
        mine.y = -1;
    }
    if (clash) mine.y = -1;                // (also a pair that copies nothing)
    src_out[i] = mine.x;
    dst_out[i] = mine.y;
}

constexpr int kCopyThreads = 128;          // warp 0 copies; the others rewrite tables (compaction)
constexpr int kFewPairs = 256;             // pairs that each CTA resolves by itself
constexpr int kCopyStages = 6;
constexpr int kCopyPiece = 16384;          // bytes of a piece at most
constexpr long long kWaitBudget = 4000000000LL;   // ~2 s of SM clock per wait

struct CopyArgs {
    unsigned char* pool[2];                // K, V
    int layers;
    size_t layer_bytes, page_bytes, row_bytes;
    int piece, pieces;                     // bytes of a piece, pieces of a page
    const int32_t* src;
    const int32_t* dst;                    // negative: nothing to copy
    const int32_t* used;                   // positions of the page to copy (null: the whole page)
    const int32_t* count;                  // pairs, on the device (null: n)
    int n;
    bool few;                              // src and dst as the caller gave them, at most kFewPairs
    // compaction: the tables that name the pages
    int32_t* block_table;
    const int32_t* row_pages;
    const int32_t* remap;
    int R, max_pages, num_pages;
    int32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const CopyArgs a)
{
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kCopyStages];
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kCopyStages; ++i) rdtc::mbar_init(&full[i], 1);
        rdtc::mbar_fence_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the pairs (and tables) are written

    __shared__ int2 pairs[kFewPairs];
    if (a.few) {
        // few pairs: every CTA finds out by itself which may be copied
        for (int i = tid; i < a.n; i += kCopyThreads) pairs[i] = pair_at(a.src, a.dst, i, a.n, a.num_pages);
        __syncthreads();
        bool clash[kFewPairs / kCopyThreads];
#pragma unroll
        for (int q = 0; q < kFewPairs / kCopyThreads; ++q) {
            const int i = tid + q * kCopyThreads;
            clash[q] = false;
            if (i >= a.n) continue;
            const int2 mine = pairs[i];
#pragma unroll 8
            for (int k = 0; k < a.n; ++k) clash[q] |= (pairs[k].y == mine.x) | ((pairs[k].y == mine.y) & (k < i));
            if (blockIdx.x == 0 && (mine.y < 0 ? pair_wrong(a.src, a.dst, i, a.num_pages) : clash[q]))
                rd_flag(a.status, RD_DEV_BAD_INDEX);
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kFewPairs / kCopyThreads; ++q)
            if (clash[q]) pairs[tid + q * kCopyThreads].y = -1;
        __syncthreads();
    }
    if (tid < 32) {
        const int lane = tid;
        const int n = a.count != nullptr ? __ldcg(a.count) : a.n;
        const long long total = (long long)n * 2 * a.layers * a.pieces;
        volatile int no_abort = 0;
        // The warp works out 32 pieces at a time, a lane each, with the pairs of the 32
        // behind them already on their way; lane 0 copies them in turn
        long long batch = blockIdx.x;                     // first piece of the batch after the one looked up
        bool looked_up = false;
        int at_page = 0, at_pool = 0, src = 0, dst = -1, used = 0;
        auto look_up = [&]() {
            looked_up = batch < total;
            const long long piece = batch + (long long)lane * gridDim.x;
            batch += 32ll * gridDim.x;
            dst = -1;
            if (piece >= total) return;
            const long long t = piece / a.pieces;
            at_page = (int)(piece - t * a.pieces);
            const int i = (int)(t / (2 * a.layers));
            at_pool = (int)(t - (long long)i * 2 * a.layers);
            src = a.few ? pairs[i].x : __ldcg(a.src + i);
            dst = a.few ? pairs[i].y : __ldcg(a.dst + i);
            if (a.used != nullptr) used = __ldcg(a.used + i);
        };
        look_up();
        unsigned left = 0u;                               // pieces of the present batch still to copy
        const unsigned char* my_from = nullptr;
        unsigned char* my_to = nullptr;
        uint32_t my_bytes = 0u;
        struct Piece { unsigned char* to; const unsigned char* from; uint32_t bytes; };
        auto take = [&](Piece& pc) -> bool {              // the next piece to copy; false: no more
            while (left == 0u) {
                if (!looked_up) return false;
                size_t bytes = a.page_bytes;
                if (a.used != nullptr) bytes = min(bytes, ((size_t)max(used, 0) * a.row_bytes + 15) & ~size_t(15));
                const size_t o = (size_t)at_page * a.piece;
                my_bytes = 0u;
                if (dst >= 0 && o < bytes) {
                    unsigned char* base = a.pool[at_pool & 1] + (size_t)(at_pool >> 1) * a.layer_bytes + o;
                    my_from = base + (size_t)src * a.page_bytes;
                    my_to = base + (size_t)dst * a.page_bytes;
                    my_bytes = (uint32_t)min((size_t)a.piece, bytes - o);
                }
                left = __ballot_sync(0xffffffffu, my_bytes > 0u);
                look_up();
            }
            const int from = __ffs((int)left) - 1;
            left &= left - 1u;
            pc.from = reinterpret_cast<const unsigned char*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(my_from), from));
            pc.to = reinterpret_cast<unsigned char*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(my_to), from));
            pc.bytes = __shfl_sync(0xffffffffu, my_bytes, from);
            return true;
        };
        unsigned char* to[kCopyStages] = {};
        uint32_t len[kCopyStages] = {};
        Piece next = {};
        bool more = take(next);                           // always one piece ahead
        uint32_t issued = 0, done = 0;
        auto load = [&](int st) {                         // the piece ahead into stage st
            to[st] = next.to;
            len[st] = next.bytes;
            if (lane == 0) {
                rdtc::mbar_arrive_expect_tx(&full[st], next.bytes);
                rdtc::bulk_load(ring + (size_t)st * a.piece, next.from, next.bytes, &full[st]);
            }
            __syncwarp();
            ++issued;
            more = take(next);
        };
        // stage st takes piece number st, st + kCopyStages, ...
#pragma unroll
        for (int st = 0; st < kCopyStages; ++st)
            if (more) load(st);
        bool ok = true;
        while (ok && done < issued) {
#pragma unroll
            for (int st = 0; st < kCopyStages; ++st) {
                if (done >= issued) break;
                const uint32_t round = done / kCopyStages;
                uint32_t landed = 1u;
                if (lane == 0) {
                    landed = rdtc::mbar_wait(&full[st], round & 1, &no_abort, kWaitBudget);
                    if (landed) {
                        rdtc::bulk_store(to[st], ring + (size_t)st * a.piece, len[st]);
                        rdtc::tma_store_commit();
                        // refill the stage before this one: its store, the last but one,
                        // has read it once at most one store is still reading
                        if (done >= 1) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    }
                }
                ok = __shfl_sync(0xffffffffu, landed, 0) != 0u;
                if (!ok) break;
                ++done;
                constexpr int before[kCopyStages] = {kCopyStages - 1, 0, 1, 2, 3, 4};
                if (done >= 2 && more) load(before[st]);
            }
        }
        if (!ok) {
            if (lane == 0) rd_flag(a.status, RD_DEV_TIMEOUT);
            // the loads in flight must land before the CTA may exit
            for (uint32_t k = done; k < issued; ++k)
                rdtc::mbar_wait(&full[k % kCopyStages], (k / kCopyStages) & 1, &no_abort, kWaitBudget);
        }
        if (lane == 0) rdtc::tma_store_wait_all();
    } else if (a.remap != nullptr && tid >= 32) {
        // table entries through the map, one row per three warps' turn
        for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
            const uint32_t h = (uint32_t)max(0, min(__ldcg(a.row_pages + r), a.max_pages));
            int32_t* row = a.block_table + (size_t)r * a.max_pages;
            for (uint32_t j = tid - 32; j < h; j += kCopyThreads - 32) {
                const int page = row[j];
                const int to = page >= 0 && page < a.num_pages ? __ldcg(a.remap + page) : -1;
                if (to < 0) rd_flag(a.status, RD_DEV_BAD_INDEX);
                else if (to != page) row[j] = to;
            }
        }
    }
}

// `dependent`: behind a kernel of the same call, which lets it start early.  The
// first kernel of a call waits for all that the stream holds.
cudaError_t launch_copy(CopyArgs& a, size_t max_pairs, bool dependent, cudaStream_t stream)
{
    const long long sms = rd_device_sm_count();
    // Pieces of 16 KB keep 2 x 6 x 16 KB in flight per SM; a copy with fewer
    // pieces than CTAs is cut finer, down to 2 KB, so that every SM takes part.
    const double bytes = (double)max_pairs * 2 * a.layers * (double)a.page_bytes;
    a.piece = kCopyPiece;
    while (a.piece > 2048 && bytes / a.piece < 4.0 * sms) a.piece /= 2;
    a.pieces = (int)((a.page_bytes + a.piece - 1) / a.piece);
    const long long total = (long long)max_pairs * 2 * a.layers * a.pieces;
    const long long want = std::max<long long>(total, a.remap != nullptr ? a.R : 0);
    const unsigned grid = (unsigned)std::max<long long>(1, std::min<long long>(want, 2 * sms));
    const int smem = kCopyStages * a.piece;
    cudaError_t e = cudaFuncSetAttribute(copy_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kCopyStages * kCopyPiece);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, copy_pages_kernel, a);
}

// One launch of a table kernel: a cluster of kTableCtas CTAs.  The limit on dynamic
// shared memory belongs to the kernel, for all host threads: it is set to what the
// largest tables take (`most`), never to what this call does (`smem`), which another
// thread's call could find too small between its setting and its launch.
constexpr size_t kResizeSmemMost = (3 * (size_t)RD_MAX_ROWS + 1) * sizeof(int);
constexpr size_t kForkSmemMost = (3 * (size_t)RD_MAX_ROWS + 1) * sizeof(int) + RD_MAX_PAGES / 8;
static_assert(kResizeSmemMost + sizeof(ScanSmem) <= 227 * 1024 && kForkSmemMost + sizeof(ScanSmem) <= 227 * 1024,
              "shared memory");
template <typename... P, typename... A>
cudaError_t launch_table(void (*kernel)(P...), size_t smem, size_t most, cudaStream_t stream, A... args)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kTableCtas);
    cfg.blockDim = dim3(kTableThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kTableCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

CopyArgs copy_args(const rd_page_pools& p, int32_t* status)
{
    CopyArgs a = {};
    a.pool[0] = static_cast<unsigned char*>(p.k_pool);
    a.pool[1] = static_cast<unsigned char*>(p.v_pool);
    a.layers = p.layers;
    a.page_bytes = p.page_bytes;
    a.layer_bytes = p.page_bytes * (size_t)p.num_pages;
    a.num_pages = p.num_pages;
    a.status = status;
    return a;
}

}  // namespace

cudaError_t rd_launch_resize_pages(int32_t* block_table, int R, int max_pages, int32_t* row_pages,
                                   int32_t* page_refs, int num_pages, const int32_t* new_lens, int page_size,
                                   int32_t* dev_status, cudaStream_t stream)
{
    const size_t smem = (size_t)(3 * R + 1) * sizeof(int);
    return launch_table(resize_kernel, smem, kResizeSmemMost, stream, block_table, R, max_pages, row_pages, page_refs,
                        num_pages, new_lens, page_size, dev_status);
}

bool rd_fork_copies_itself(int n, int layers, size_t page_bytes)
{
    return (double)n * 2 * layers * (double)page_bytes <= (double)kForkHereBytes;
}

cudaError_t rd_launch_fork_pages(const rd_page_pools& pools, int page_size, int32_t* block_table, int R,
                                 int max_pages, int32_t* row_pages, int32_t* page_refs, int32_t* ctx_lens,
                                 const int32_t* parent, const int32_t* child, int n, void* workspace,
                                 int32_t* dev_status, cudaStream_t stream)
{
    const bool here = rd_fork_copies_itself(n, pools.layers, pools.page_bytes);
    int32_t* src = here ? nullptr : static_cast<int32_t*>(workspace);
    int32_t* dst = here ? nullptr : src + n;
    int32_t* used = here ? nullptr : dst + n;
    ForkCopy fc = {};
    if (here) {
        fc.pool[0] = static_cast<uint4*>(pools.k_pool);
        fc.pool[1] = static_cast<uint4*>(pools.v_pool);
        fc.layers = pools.layers;
        fc.page_vecs = pools.page_bytes / 16;
        fc.layer_vecs = fc.page_vecs * (size_t)pools.num_pages;
        fc.row_bytes = pools.page_bytes / page_size;
    }
    const size_t smem =
        (size_t)(2 * n + 1 + R + words_per_warp(pools.num_pages) * kTableCtas * kTableWarps) * sizeof(int);
    cudaError_t e = launch_table(fork_kernel, smem, kForkSmemMost, stream, block_table, R, max_pages, row_pages,
                                 page_refs, pools.num_pages, ctx_lens, parent, child, n, page_size, src, dst, used, fc,
                                 dev_status);
    if (e != cudaSuccess || here) return e;
    CopyArgs a = copy_args(pools, dev_status);
    a.row_bytes = pools.page_bytes / page_size;
    a.src = src;
    a.dst = dst;
    a.used = used;
    a.n = n;
    return launch_copy(a, n, true, stream);
}

// comparing every pair with every other in each CTA takes a microsecond at 256
bool rd_copy_resolves_itself(int n) { return n <= kFewPairs; }

cudaError_t rd_launch_copy_pages(const rd_page_pools& pools, const int32_t* src, const int32_t* dst, int n,
                                 void* workspace, int32_t* dev_status, cudaStream_t stream)
{
    CopyArgs a = copy_args(pools, dev_status);
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.few = rd_copy_resolves_itself(n);
    if (!a.few) {
        int32_t* rs = static_cast<int32_t*>(workspace);
        int32_t* rt = rs + n;
        resolve_kernel<<<(n + kResolveThreads - 1) / kResolveThreads, kResolveThreads, 0, stream>>>(
            src, dst, n, pools.num_pages, rs, rt, dev_status);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        a.src = rs;
        a.dst = rt;
    }
    return launch_copy(a, n, !a.few, stream);
}

cudaError_t rd_launch_compact_pages(const rd_page_pools& pools, int32_t* block_table, int R, int max_pages,
                                    const int32_t* row_pages, int32_t* page_refs, int32_t* remap,
                                    int32_t* n_live, void* workspace, int32_t* dev_status, cudaStream_t stream)
{
    // at most half of the pages move: a hole below n_live for each
    const int most = pools.num_pages / 2;
    int32_t* n_moves = static_cast<int32_t*>(workspace);
    int32_t* src = n_moves + 4;
    int32_t* dst = src + most;
    cudaError_t e = launch_table(compact_plan_kernel, 0, 0, stream, page_refs, pools.num_pages, remap, n_live, n_moves,
                                 src, dst);
    if (e != cudaSuccess) return e;
    CopyArgs a = copy_args(pools, dev_status);
    a.src = src;
    a.dst = dst;
    a.count = n_moves;
    a.block_table = block_table;
    a.row_pages = row_pages;
    a.remap = remap;
    a.R = R;
    a.max_pages = max_pages;
    return launch_copy(a, most, true, stream);
}
