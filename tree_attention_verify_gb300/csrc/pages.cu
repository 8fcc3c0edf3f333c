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
//  - the page copy: bulk copies (TMA) through a shared-memory ring, one issuing
//    thread per CTA, two CTAs per SM; a page of K or V is one contiguous block,
//    so nothing but the ring's depth and HBM bounds it.
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

__device__ __forceinline__ PageWords read_free(const int32_t* refs, int num_pages, int rank)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (num_pages + 31) / 32;
    PageWords p;
    p.q = (words + kTableCtas * kTableWarps - 1) / (kTableCtas * kTableWarps);
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
    __shared__ ScanSmem sc;
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const int warp = rank * kTableWarps + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;

    auto wanted = [&](int r, int h) {      // pages of row r after the call
        const int n = __ldg(new_lens + r);
        if (n < 0) return h;
        const int w = n == 0 ? 0 : (n - 1) / page_size + 1;
        return w;
    };
    const int demand = cta_scan_array(R, off, sc.warp_sum, [&](int r) {
        int h = __ldcg(row_pages + r);
        const int w = wanted(r, h);
        if (h < 0 || h > max_pages || w > max_pages) {
            if (rank == 0) rd_flag(status, RD_DEV_BAD_LENGTH);
            h = -1;
        }
        have[r] = h;
        return h < 0 ? 0 : max(0, w - h);
    });
    // give pages back
    for (int r = warp; r < R; r += kTableCtas * kTableWarps) {
        const int h = have[r];
        if (h < 0) continue;
        int32_t* row = block_table + (size_t)r * max_pages;
        for (int j = wanted(r, h) + lane; j < h; j += 32) {
            const int page = row[j];
            row[j] = -1;
            if (page < 0 || page >= num_pages) {
                rd_flag(status, RD_DEV_BAD_INDEX);
            } else if (atomicSub(refs + page, 1) <= 0) {        // held by nobody: leave it free
                atomicAdd(refs + page, 1);
                rd_flag(status, RD_DEV_BAD_INDEX);
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
        else row_pages[r] = wanted(r, h);
    }
}

// Rows branch: tables here, the last pages' data by the copy kernel behind it.
__global__ void __launch_bounds__(kTableThreads, 1)
fork_kernel(int32_t* block_table, int R, int max_pages, int32_t* row_pages, int32_t* refs, int num_pages,
            int32_t* ctx_lens, const int32_t* __restrict__ parent, const int32_t* __restrict__ child, int n,
            int page_size, int32_t* src, int32_t* dst, int32_t* used, int32_t* status)
{
    extern __shared__ int dyn[];
    int* off = dyn;                        // [n + 1] new pages of the pairs before
    int* len = dyn + n + 1;                // [n] the parent's length, -1: no pair
    int* owner = len + n;                  // [R] first pair that names the row as its child
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
    if (rank == 0)
        for (int i = tid; i < n; i += kTableThreads) dst[i] = -1;
    // every CTA has read the tables before any is changed
    cl.sync();
    int n_free;
    const PageWords p = read_free(refs, num_pages, rank);
    const int base = cluster_rank(p.bits, sc, cl, n_free);
    for_ranked(p, p.bits, base, min(demand, n_free), [&](int page, int k) {
        const int i = last_at_most(off, n, k);
        const int full = len[i] / page_size;
        const int from = __ldcg(block_table + (size_t)__ldg(parent + i) * max_pages + full);
        block_table[(size_t)__ldg(child + i) * max_pages + full] = page;
        refs[page] = 1;
        if (from < 0 || from >= num_pages) {
            rd_flag(status, RD_DEV_BAD_INDEX);                  // nothing to copy
            return;
        }
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
        for (int j = lane; j < full; j += 32) {
            const int page = __ldcg(block_table + (size_t)from * max_pages + j);
            block_table[(size_t)to * max_pages + j] = page;
            if (page < 0 || page >= num_pages) rd_flag(status, RD_DEV_BAD_INDEX);
            else atomicAdd(refs + page, 1);
        }
        if (lane == 0) {
            row_pages[to] = full + (off[i + 1] - off[i]);
            ctx_lens[to] = l;
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
__global__ void __launch_bounds__(kResolveThreads)
resolve_kernel(const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, int num_pages,
               int32_t* src_out, int32_t* dst_out, int32_t* status)
{
    __shared__ int2 tile[kResolveThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int i = blockIdx.x * kResolveThreads + threadIdx.x;
    auto load = [&](int k) {               // (-1, -1): copies nothing
        int2 v = make_int2(-1, -1);
        if (k < n) {
            v = make_int2(__ldg(src + k), __ldg(dst + k));
            if (v.x < 0 || v.x >= num_pages || v.y < 0 || v.y >= num_pages || v.x == v.y) v = make_int2(-1, -1);
        }
        return v;
    };
    int2 mine = load(i);
    bool clash = false;
    for (int k0 = 0; k0 < n; k0 += kResolveThreads) {
        __syncthreads();
        tile[threadIdx.x] = load(k0 + threadIdx.x);
        __syncthreads();
        const int m = min(kResolveThreads, n - k0);
        for (int k = 0; k < m; ++k) {
            const int d = tile[k].y;
            clash = clash || (d >= 0 && (d == mine.x || (d == mine.y && k0 + k < i)));
        }
    }
    if (i >= n) return;
    if (mine.y < 0) {
        const int s = __ldg(src + i), d = __ldg(dst + i);
        if (s >= num_pages || (s >= 0 && s != d)) rd_flag(status, RD_DEV_BAD_INDEX);
    } else if (clash) {
        rd_flag(status, RD_DEV_BAD_INDEX);
        mine.y = -1;
    }
    src_out[i] = mine.x;
    dst_out[i] = mine.y;
}

constexpr int kCopyThreads = 128;          // thread 0 copies; the others rewrite tables (compaction)
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
    // compaction: the tables that name the pages
    int32_t* block_table;
    const int32_t* row_pages;
    const int32_t* remap;
    int R, max_pages, num_pages;
    int32_t* status;
};

__device__ __forceinline__ void bulk_load(void* smem, const void* gmem, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(rdtc::smem_addr(smem)), "l"(gmem), "r"(bytes), "r"(rdtc::smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void bulk_store(void* gmem, const void* smem, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 ::"l"(gmem), "r"(rdtc::smem_addr(smem)), "r"(bytes) : "memory");
}

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

    if (tid == 0) {
        const int n = a.count != nullptr ? __ldcg(a.count) : a.n;
        const long long total = (long long)n * 2 * a.layers * a.pieces;
        volatile int no_abort = 0;
        long long next = blockIdx.x;
        // the next piece to copy from `next` on; false: no more
        struct Piece { unsigned char* to; const unsigned char* from; uint32_t bytes; };
        auto take = [&](Piece& pc) -> bool {
            for (; next < total; next += gridDim.x) {
                const int k = (int)(next % a.pieces);
                const long long t = next / a.pieces;
                const int kl = (int)(t % (2 * a.layers)), i = (int)(t / (2 * a.layers));
                const int s = __ldcg(a.src + i), d = __ldcg(a.dst + i);
                if (d < 0) continue;
                size_t bytes = a.page_bytes;
                if (a.used != nullptr) bytes = min(bytes, ((size_t)__ldcg(a.used + i) * a.row_bytes + 15) & ~size_t(15));
                const size_t o = (size_t)k * a.piece;
                if (o >= bytes) continue;
                unsigned char* base = a.pool[kl & 1] + (size_t)(kl >> 1) * a.layer_bytes + o;
                pc.from = base + (size_t)s * a.page_bytes;
                pc.to = base + (size_t)d * a.page_bytes;
                pc.bytes = (uint32_t)min((size_t)a.piece, bytes - o);
                next += gridDim.x;
                return true;
            }
            return false;
        };
        Piece held[kCopyStages];
        uint32_t issued = 0, done = 0;
        bool more = true;
        // stage st takes piece number st, st + kCopyStages, ...
#pragma unroll
        for (int st = 0; st < kCopyStages; ++st) {
            if (more && (more = take(held[st]))) {
                rdtc::mbar_arrive_expect_tx(&full[st], held[st].bytes);
                bulk_load(ring + (size_t)st * a.piece, held[st].from, held[st].bytes, &full[st]);
                ++issued;
            }
        }
        bool ok = true;
        while (ok && done < issued) {
#pragma unroll
            for (int st = 0; st < kCopyStages; ++st) {
                if (done >= issued) break;
                const uint32_t round = done / kCopyStages;
                if (!rdtc::mbar_wait(&full[st], round & 1, &no_abort, kWaitBudget)) { ok = false; break; }
                bulk_store(held[st].to, ring + (size_t)st * a.piece, held[st].bytes);
                rdtc::tma_store_commit();
                ++done;
                // refill the stage before this one: its store, the last but one, has
                // read it once at most one store is still reading
                if (done >= 2 && more) {
                    const int ps = (st + kCopyStages - 1) % kCopyStages;
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    if ((more = take(held[ps]))) {
                        rdtc::mbar_arrive_expect_tx(&full[ps], held[ps].bytes);
                        bulk_load(ring + (size_t)ps * a.piece, held[ps].from, held[ps].bytes, &full[ps]);
                        ++issued;
                    }
                }
            }
        }
        if (!ok) {
            rd_flag(a.status, RD_DEV_TIMEOUT);
            // the loads in flight must land before the CTA may exit
            for (uint32_t k = done; k < issued; ++k)
                rdtc::mbar_wait(&full[k % kCopyStages], (k / kCopyStages) & 1, &no_abort, kWaitBudget);
        }
        rdtc::tma_store_wait_all();
    } else if (a.remap != nullptr && tid >= 32) {
        // table entries through the map, one row per three warps' turn
        for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
            const int h = min(__ldcg(a.row_pages + r), a.max_pages);
            int32_t* row = a.block_table + (size_t)r * a.max_pages;
            for (int j = tid - 32; j < h; j += kCopyThreads - 32) {
                const int page = row[j];
                const int to = page >= 0 && page < a.num_pages ? __ldcg(a.remap + page) : -1;
                if (to < 0) rd_flag(a.status, RD_DEV_BAD_INDEX);
                else if (to != page) row[j] = to;
            }
        }
    }
}

cudaError_t launch_copy(CopyArgs& a, size_t max_pairs, cudaStream_t stream)
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_pages_kernel, a);
}

// One launch of a table kernel: a cluster of kTableCtas CTAs.
template <typename... P, typename... A>
cudaError_t launch_table(void (*kernel)(P...), size_t smem, cudaStream_t stream, A... args)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
    const size_t smem = (size_t)(2 * R + 1) * sizeof(int);
    return launch_table(resize_kernel, smem, stream, block_table, R, max_pages, row_pages, page_refs, num_pages,
                        new_lens, page_size, dev_status);
}

cudaError_t rd_launch_fork_pages(const rd_page_pools& pools, int page_size, int32_t* block_table, int R,
                                 int max_pages, int32_t* row_pages, int32_t* page_refs, int32_t* ctx_lens,
                                 const int32_t* parent, const int32_t* child, int n, void* workspace,
                                 int32_t* dev_status, cudaStream_t stream)
{
    int32_t* src = static_cast<int32_t*>(workspace);
    int32_t* dst = src + n;
    int32_t* used = dst + n;
    const size_t smem = (size_t)(2 * n + 1 + R) * sizeof(int);
    cudaError_t e = launch_table(fork_kernel, smem, stream, block_table, R, max_pages, row_pages, page_refs,
                                 pools.num_pages, ctx_lens, parent, child, n, page_size, src, dst, used, dev_status);
    if (e != cudaSuccess) return e;
    CopyArgs a = copy_args(pools, dev_status);
    a.row_bytes = pools.page_bytes / page_size;
    a.src = src;
    a.dst = dst;
    a.used = used;
    a.n = n;
    return launch_copy(a, n, stream);
}

cudaError_t rd_launch_copy_pages(const rd_page_pools& pools, const int32_t* src, const int32_t* dst, int n,
                                 void* workspace, int32_t* dev_status, cudaStream_t stream)
{
    int32_t* rs = static_cast<int32_t*>(workspace);
    int32_t* rt = rs + n;
    resolve_kernel<<<(n + kResolveThreads - 1) / kResolveThreads, kResolveThreads, 0, stream>>>(
        src, dst, n, pools.num_pages, rs, rt, dev_status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    CopyArgs a = copy_args(pools, dev_status);
    a.src = rs;
    a.dst = rt;
    a.n = n;
    return launch_copy(a, n, stream);
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
    cudaError_t e = launch_table(compact_plan_kernel, 0, stream, page_refs, pools.num_pages, remap, n_live, n_moves,
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
    return launch_copy(a, most, stream);
}
