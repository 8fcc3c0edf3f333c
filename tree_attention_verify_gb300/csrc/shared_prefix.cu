// rd_tree_attention_shared: tree attention over a paged cache for a batch whose
// groups of requests share a long prefix, the prefix read once per group.
//
// Softmax attention splits over its keys: with partials
//   m_i = max_k s_k, l_i = sum_k 2^(s_k - m_i), O_i = sum_k 2^(s_k - m_i) v_k
// over disjoint key sets i, the output is sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// with M = max_i m_i.  So the prefix of a group is one dense product of all its
// requests' rows with the shared keys, and the rest of each request is the
// paged tree attention from behind the prefix.  On one stream, each launch a
// programmatic dependent of the one before:
//   plan    one CTA: valid requests, the compact list of a group's live rows,
//           and the table that divides the prefix work over the CTAs;
//   prefix  (below) fp32 partials of every live row over its group's prefix;
//   suffix  partials of every row over its request's own context and drafts
//           (shared_suffix.cu for up to 128 rows per kv head, else the shared-prefix
//           variant of attention_tc.cu);
//   merge   the formula above, rounded once to bf16; zeros in padded rows.  With many
//           units the suffix kernel ends each in this way itself.
//
// The prefix kernel: unit = (group, kv head, 256 rows), the rows being the G
// query heads of each live node of the group, in request order.  One CTA per SM
// with two 128-row tiles, K and V in chunks of 128 positions.  Every position is
// visible to every row (whole pages), so there is no mask at all.  The units'
// chunks form one sequence that the CTAs take in equal ranges, so that one group
// with few rows still fills the GPU; a unit cut by a range boundary leaves its
// pieces to the merge.
// Warp roles (640 threads):
//   warps 0-15  softmax: a warpgroup for each half (64 positions) of each tile's
//              chunk; row r is TMEM lane r of both.  S from TMEM, online softmax in
//              exp2 form, bf16 P written over S.  A row's two threads share its
//              running maximum, and only a chunk in which some row's grows by more
//              than 2^8 makes them exchange it and rescale O; one reducing barrier
//              a chunk tells.  (One warpgroup a tile had the tensor core wait: its
//              1,900 cycles a chunk and the 768 of the products behind it come one
//              after the other.)
//   warp 16    producer: K_0, V_0, K_1, V_1, ... by TMA into one ring
//   warp 17    MMA issuer: per chunk j and tile t, O_t += P_t V_j, then S_t of
//              chunk j + 1, so that the tensor core works on one tile while the
//              other's softmax runs
//   warps 18-19  the unit's query rows into shared memory (cp.async, row list),
//              then the check that a group's tables name the same pages
// What bounds it: with many rows the chain S -> softmax -> P -> PV of a tile (64
// requests of 23 live nodes, 40 heads, 8,192 positions: 244 GFLOP in 170 us, 1.44 PFLOP/s,
// tensor pipe active 63% of the time; L2 misses on K and V cost 4% of it, measured by
// reading one head's K and V for all), with few rows the start and end of a unit.
// Every wait is bounded by a clock budget; on expiry the CTA records
// RD_DEV_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "block_scan.cuh"
#include "rd_internal.cuh"
#include "shared_prefix.cuh"
#include "tc_ptx.cuh"

namespace {
using namespace rdtc;
using namespace rdattn;
using namespace rdshared;

constexpr int kM = 128;                    // rows per tile = TMEM lanes
static_assert(kUnitRows == 2 * kM, "two tiles");
constexpr int kN = 128;                    // KV positions per chunk (two TMA boxes)
constexpr int kSoftmaxWarps = 16;          // four warpgroups: (tile, half)
constexpr int kThreads = kSoftmaxWarps * 32 + 128;
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
constexpr int kQWarp0 = 18;                // two query warps
// 640 threads leave 96 registers each: the softmax warps read their scores twice,
// 32 at a time, rather than hold half a row (64) over the barrier between.
// Division over the CTAs, in eighths of a chunk of two tiles.  A chunk of one tile (a
// unit of at most 128 rows) takes five; beginning a unit (its queries, the first
// scores, the last sums) takes a CTA as long as three chunks.  At 320 units on 152
// CTAs, equal numbers of chunks left the slowest CTA 22% behind the fastest.
constexpr uint32_t kTwoTiles = 8;
constexpr uint32_t kOneTile = 5;
constexpr uint32_t kUnitStart = 24;
// A CTA's share at least: 2, 3 and 4 chunks make 8 single tokens over 2,048 positions
// 22.6, 23.0 and 25.5 us, 4 requests of 20 nodes (10 of them live) 28.9, 28.3 and 26.7.
constexpr uint32_t kMinRange = 3 * kTwoTiles;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr long long kWaitBudget = 4000000000LL;   // ~2 s of SM clock per wait

// What the units of one kv head of a group count in the division.
struct UnitCost {
    uint32_t n;               // chunks of a unit
    uint32_t full, head;      // a unit of two tiles, all units of a kv head
    uint32_t last;            // weight of a chunk of the last unit
    __device__ __forceinline__ UnitCost(const Group& g, int G)
    {
        n = (uint32_t)(g.positions + kN - 1) / kN;
        full = kUnitStart + kTwoTiles * n;
        last = g.nodes * G - (g.pairs - 1) * kUnitRows <= kM ? kOneTile : kTwoTiles;
        head = (uint32_t)(g.pairs - 1) * full + kUnitStart + last * n;
    }
};

// ------------------------------------------------------------------------ plan
struct PlanArgs {
    int B, P_max, Hkv, G, page_size, max_pages, max_ctx, n_groups;
    int suffix_chunk;          // positions of a suffix chunk (0: the tcgen05 kernel divides by itself)
    int suffix_nodes;          // nodes of a suffix unit
    const int32_t* lens;
    const int32_t* ctx_lens;
    const int32_t* group_offsets;
    const int32_t* prefix_pages;
    Plan p;
    int32_t* status;
};

// A short chain of dependent reads is all this kernel is, so a batch of up to 1024
// requests and groups (kSmall) keeps its tables in shared memory between the steps;
// a larger one reads them back from the workspace.
template <bool kSmall>
__global__ void __launch_bounds__(kScanThreads, 1)
plan_kernel(const PlanArgs a)
{
    constexpr int kCap = kSmall ? kScanThreads : 1;
    __shared__ int warp_sum[kScanWarps];
    __shared__ int s_offsets[kCap + 1], s_pages[kCap], s_base[kCap + 1];
    __shared__ Group s_group[kCap];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t* offsets = a.group_offsets;
    const int32_t* pages = a.prefix_pages;
    int32_t* base = a.p.node_base;
    Group* group = a.p.group;
    int ctx = 0, len = 0;                                  // kSmall: of request tid
    if constexpr (kSmall) {
        if (tid < a.B) {
            ctx = __ldg(a.ctx_lens + tid);
            len = __ldg(a.lens + tid);
        }
        for (int g = tid; g <= a.n_groups; g += kScanThreads) s_offsets[g] = __ldg(offsets + g);
        if (tid < a.n_groups) s_pages[tid] = __ldg(pages + tid);
        offsets = s_offsets;
        pages = s_pages;
        base = s_base;
        group = s_group;
        __syncthreads();
    }
    // offsets that do not ascend within [0, B] would give a request two groups:
    // then nobody shares (the results stay the same)
    bool bad_offsets = false;
    for (int g = tid; g < a.n_groups; g += kScanThreads) {
        const int o0 = offsets[g], o1 = offsets[g + 1];
        bad_offsets = bad_offsets || o0 < 0 || o1 < o0 || o1 > a.B;
    }
    bad_offsets = __syncthreads_or(bad_offsets);
    if (bad_offsets && tid == 0) rd_flag(a.status, RD_DEV_BAD_INDEX);
    auto pages_of = [&](int g) {
        const int n = pages[g];
        return n < 0 || n > a.max_pages || (long long)n * a.page_size > a.max_ctx ? -1 : n;
    };
    int carry = 0, my_gid = -1;
    uint32_t suf_carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kScanThreads) {
        const int b = b0 + tid;
        int n = 0, suf = 0;
        if (b < a.B) {
            int g = -1, skip = 0;
            if (!bad_offsets) {
                int lo = 0, hi = a.n_groups;               // groups that start at or before b
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (offsets[mid] <= b) lo = mid + 1; else hi = mid;
                }
                if (lo > 0 && b < offsets[lo]) {
                    const int pg = pages_of(lo - 1);
                    if (pg > 0) {
                        g = lo - 1;
                        skip = pg * a.page_size;
                    }
                }
            }
            if constexpr (!kSmall) {
                ctx = a.ctx_lens[b];
                len = a.lens[b];
            }
            if (ctx < (len > 0 ? skip : 0) || ctx > a.max_ctx || ctx > kRdMaxContext ||
                (long long)ctx > (long long)a.max_pages * a.page_size || len < 0 || len > a.P_max) {
                rd_flag(a.status, RD_DEV_BAD_LENGTH);
                len = 0;
            }
            if (len == 0) {                                // no rows: of no group, its table is not read
                g = -1;
                skip = 0;
            }
            a.p.eff_len[b] = len;
            a.p.skip[b] = skip;
            a.p.gid[b] = my_gid = g;
            n = g >= 0 ? len : 0;
            if (a.suffix_chunk > 0 && len > 0)
                suf = a.Hkv * ((len + a.suffix_nodes - 1) / a.suffix_nodes) *
                      ((ctx - skip + a.suffix_chunk - 1) / a.suffix_chunk + (len + a.suffix_chunk - 1) / a.suffix_chunk);
        }
        int total;
        const int at = carry + cta_scan(n, warp_sum, total);
        if (b < a.B) {
            base[b] = at;
            for (int p = 0; p < n; ++p) a.p.node_row[at + p] = b * a.P_max + p;
        }
        carry += total;
        if (a.suffix_chunk > 0) {
            const int before = cta_scan(suf, warp_sum, total);
            if (b < a.B) a.p.suf_first[b] = suf_carry + before;
            suf_carry += total;
        }
    }
    if (tid == 0) {
        base[a.B] = carry;
        if (a.suffix_chunk > 0) a.p.suf_first[a.B] = suf_carry;
    }
    __syncthreads();
    uint32_t chunks = 0;
    int all_units = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += kScanThreads) {
        const int g = g0 + tid;
        int w = 0, units = 0;
        Group grp = {0, 0, 0, 0, 0, 0};
        if (g < a.n_groups && !bad_offsets) {
            const int pg = pages_of(g);
            if (pg < 0) rd_flag(a.status, RD_DEV_BAD_LENGTH);
            grp.leader = offsets[g];
            grp.node0 = base[grp.leader];
            grp.nodes = base[offsets[g + 1]] - grp.node0;
            if (grp.nodes > 0) {
                // the first with rows: the last before which there are none
                int lo = grp.leader, hi = offsets[g + 1] - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (base[mid] == grp.node0) lo = mid; else hi = mid - 1;
                }
                grp.leader = lo;
            }
            grp.positions = max(0, pg) * a.page_size;
            grp.pairs = (grp.nodes * a.G + kUnitRows - 1) / kUnitRows;
            units = a.Hkv * grp.pairs;
            w = grp.positions > 0 && grp.nodes > 0 ? a.Hkv * (int)UnitCost(grp, a.G).head : 0;
        }
        int total, total_units;
        const int at = cta_scan(w, warp_sum, total);
        grp.unit0 = all_units + cta_scan(units, warp_sum, total_units);
        if (g < a.n_groups) {
            a.p.group[g] = grp;
            if constexpr (kSmall) s_group[g] = grp;
            a.p.first[g] = chunks + at;
        }
        chunks += total;
        all_units += total_units;
    }
    if (tid == 0) {
        a.p.first[a.n_groups] = chunks;
        *a.p.suf_next = 0;
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kScanThreads) {
        const int g = kSmall ? my_gid : a.p.gid[b];
        int4 req = make_int4(-1, 0, 0, 0);
        if (g >= 0) {
            const Group grp = group[g];
            const int node = base[b];
            req = make_int4(grp.unit0, grp.pairs, (node - grp.node0) * a.G, node * a.G);
        }
        a.p.req[b] = req;
    }
}

// ---------------------------------------------------------------------- prefix
template <int D> struct Cfg {
    static constexpr int kDB = D / 64;                  // 128-byte column blocks
    static constexpr int kStageBytes = kN * D * 2;      // one chunk of K or of V
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kQBytes = kM * D * 2;          // one tile's queries
    static constexpr int kQOff = kStages * kStageBytes;
    static constexpr int kBarOff = kQOff + 2 * kQBytes;
    static constexpr int kShareOff = kBarOff + 512;           // a float per row: what a row's two threads exchange
    static constexpr int kSmemBytes = kShareOff + 1024 + 1024;   // + alignment slack
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    // TMEM (512 columns): S of tile t (P of each half of the positions over the first
    // half of its scores), O of tile t
    static constexpr uint32_t kTmemCols = 512;
    __host__ __device__ static constexpr uint32_t s_col(int t) { return 128u * t; }
    __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + 128u * t; }
};

struct PrefixArgs {
    int B, Hq, Hkv, G, page_size, max_pages, num_pages, n_groups;
    float scale_log2;
    const uint16_t* q;                     // [B P_max, Hq, D]
    const int32_t* block_table;
    Plan p;
    int32_t* status;
    long long stall_budget;                // failure-detection test hook
};

struct Bar {
    uint64_t kv_full[8];
    uint64_t kv_empty[8];
    uint64_t q_full;          // the unit's query tiles are in shared memory
    uint64_t q_free;          // every S MMA of the unit has completed
    uint64_t s_full[2];       // S of the tile's chunk is in TMEM (and PV of the one before is done)
    uint64_t p_full[2];       // P of the tile's chunk is written (eight softmax warps)
    uint64_t o_final[2];      // the tile's last PV of the unit has completed
    uint64_t o_free[2];       // the tile's epilogue has read O
    uint64_t drain;
    uint64_t never;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bar) <= 512, "barrier block");

// One piece of a unit (all of it, unless cut).
struct Piece {
    int h, row0;              // kv head; first row of the unit within its group
    int rows;                 // rows of the unit (1 .. 256)
    int c0, n;                // chunks [c0, c0 + n)
    int slot;                 // piece slot, -1: a whole unit
    int unit;
    uint32_t last;            // where the unit's last chunk begins in the sequence
    Group g;
};

// This CTA's range of the sequence, in pieces.  A unit is its start, then its
// chunks; a chunk belongs to the CTA whose range holds its first eighth.
struct Walk {
    uint32_t x, end;
    bool first;               // no piece yet
    __device__ __forceinline__ void begin(const PrefixArgs& a)
    {
        const uint32_t W = a.p.first[a.n_groups];
        x = end = 0u;
        first = true;
        if (W == 0u) return;
        const uint32_t n = range_ctas(W, gridDim.x, kMinRange);
        if (blockIdx.x >= n) return;
        x = range_start(W, n, blockIdx.x);
        end = range_start(W, n, blockIdx.x + 1);
    }
    __device__ __forceinline__ bool next(const PrefixArgs& a, Piece& u)
    {
        while (x < end) {
            int lo = 0, hi = a.n_groups - 1;                // last group with first <= x
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.p.first[mid] <= x) lo = mid; else hi = mid - 1;
            }
            u.g = a.p.group[lo];
            const UnitCost cost(u.g, a.G);
            const uint32_t base = a.p.first[lo];
            const uint32_t h = (x - base) / cost.head;
            const uint32_t pair = min((x - base - h * cost.head) / cost.full, (uint32_t)u.g.pairs - 1);
            const uint32_t u0 = base + h * cost.head + pair * cost.full;
            const uint32_t w = pair + 1 == (uint32_t)u.g.pairs ? cost.last : kTwoTiles;
            const uint32_t at = u0 + kUnitStart;            // its first chunk
            const uint32_t stop = min(at + w * cost.n, end);
            const uint32_t c0 = x > at ? (x - at + w - 1) / w : 0u;
            const uint32_t c1 = stop > at ? (stop - at + w - 1) / w : 0u;
            x = stop;
            if (c1 <= c0) continue;                         // no chunk's first eighth
            u.h = (int)h;
            u.row0 = (int)pair * kUnitRows;
            u.rows = min(kUnitRows, u.g.nodes * a.G - u.row0);
            u.c0 = (int)c0;
            u.n = (int)(c1 - c0);
            u.slot = c1 - c0 == cost.n ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1);
            u.unit = u.g.unit0 + (int)(h * u.g.pairs + pair);
            u.last = at + w * (cost.n - 1);
            first = false;
            return true;
        }
        return false;
    }
};

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem) : "memory");
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// OR of a predicate over `count` threads at named barrier `id` (0 is __syncthreads)
__device__ __forceinline__ bool barrier_or(int id, int count, bool p)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"(count), "r"((uint32_t)p) : "memory");
    return r != 0;
}

// two floats in one 64-bit register pair (first: low half)
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefix_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v)
{
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bar& bar = *reinterpret_cast<Bar*>(smem + C::kBarOff);
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bar.abort;
    volatile int no_abort = 0;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bar.kv_full[i], 1);
            mbar_init(&bar.kv_empty[i], 1);
        }
        mbar_init(&bar.q_full, 2);
        mbar_init(&bar.q_free, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar.s_full[t], 1);
            mbar_init(&bar.p_full[t], 8);
            mbar_init(&bar.o_final[t], 1);
            mbar_init(&bar.o_free[t], 8);
        }
        mbar_init(&bar.drain, 1);
        mbar_init(&bar.never, 1);
        bar.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bar.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the plan is written
    // the suffix kernel may start (it reads the plan, and waits for this grid before
    // it reads the partials)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto fail = [&]() {
        *abort = 1;
        rd_flag(a.status, RD_DEV_TIMEOUT);
    };

    if (warp >= kSoftmaxWarps) {
    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            uint32_t g = 0;                               // ring entries issued
            Walk w;
            w.begin(a);
            Piece u;
            const uint32_t W = a.p.first[a.n_groups];
            while (!*abort && w.next(a, u)) {
                if (u.c0 == 0) {                          // the unit starts here: name its pieces
                    const uint32_t nc = range_ctas(W, gridDim.x, kMinRange);
                    const int n = u.slot < 0 ? 1 : (int)(range_of(W, nc, u.last) - blockIdx.x) + 1;
                    a.p.unit[u.unit] = make_int2(n, u.slot);
                }
                const int32_t* table = a.block_table + (size_t)u.g.leader * a.max_pages;
                auto row_of = [&](int pos) -> int {       // pool row of a position of the prefix
                    int pg = __ldg(table + pos / a.page_size);
                    if (pg < 0 || pg >= a.num_pages) {
                        rd_flag(a.status, RD_DEV_BAD_INDEX);
                        pg = 0;
                    }
                    return pg * a.page_size + pos % a.page_size;
                };
                // the rows of a chunk's two halves, looked up one chunk ahead
                auto rows_of = [&](int c, int (&z)[2]) {
                    const int pos = c * kN;
                    z[0] = row_of(pos);
                    z[1] = pos + 64 < u.g.positions ? row_of(pos + 64) : -1;
                };
                int z[2], nz[2];
                rows_of(u.c0, nz);
                bool ok = true;
                for (int j = 0; ok && j < u.n; ++j) {
                    z[0] = nz[0];
                    z[1] = nz[1];
                    if (j + 1 < u.n) rows_of(u.c0 + j + 1, nz);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++g) {
                        const int st = (int)(g % C::kStages);
                        if (g >= (uint32_t)C::kStages &&
                            !mbar_wait(&bar.kv_empty[st], ((g / C::kStages) - 1) & 1, abort, kWaitBudget)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bar.kv_full[st], z[1] >= 0 ? C::kStageBytes : C::kStageBytes / 2);
                        unsigned char* dst = smem + st * C::kStageBytes;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (z[half] < 0) continue;
#pragma unroll
                            for (int db = 0; db < C::kDB; ++db)
                                tma_load_3d(dst + db * (kN * 128) + half * (64 * 128), kv ? &map_v : &map_k,
                                            &bar.kv_full[st], db * 64, u.h, z[half]);
                        }
                    }
                }
                if (!ok) { fail(); break; }
            }
            // drain: every issued copy must land before the CTA may exit
            for (uint32_t k = g > (uint32_t)C::kStages ? g - C::kStages : 0u; k < g; ++k)
                mbar_wait(&bar.kv_full[k % C::kStages], (k / C::kStages) & 1, &no_abort, kWaitBudget);
        }
    } else if (warp >= kQWarp0) {
        // ------------------------------------------------------- query loader
        // Warp t loads tile t.  Row m of the unit is head row % G of compact node
        // row / G; a lane looks four rows up while the tile before is still in use,
        // then half a warp copies a row in 16-byte pieces (cp.async), all 128 rows'
        // in flight at once.  Rows past the unit's are zero.
        constexpr int kVecs = D / 8;                      // 16-byte pieces of a row
        constexpr int kRowsAtOnce = 32 / kVecs;
        const int t0 = tid - kQWarp0 * 32;                // 0 .. 63
        const int t = warp - kQWarp0;
        uint32_t it = 0;
        Walk w;
        w.begin(a);
        Piece u;
        while (!*abort && w.next(a, u)) {
            const bool active = t == 0 || u.rows > kM;
            uint32_t at[4];                               // row of q, of tile rows lane + 32 k
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int m = t * kM + lane + 32 * k, row = u.row0 + m;
                at[k] = 0xffffffffu;
                if (m < u.rows)
                    at[k] = (uint32_t)__ldcg(a.p.node_row + u.g.node0 + row / a.G) * a.Hq + u.h * a.G + row % a.G;
            }
            if (it > 0 && !warp_wait(&bar.q_free, (it - 1) & 1, abort, kWaitBudget)) { fail(); break; }
            if (active) {
                const int c = lane % kVecs;
                unsigned char* base = smem + C::kQOff + t * C::kQBytes + (c >> 3) * (kM * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll 2
                    for (int i = 0; i < 32; i += kRowsAtOnce) {
                        const int m = i + lane / kVecs;
                        const uint32_t row = __shfl_sync(0xffffffffu, at[k], m);
                        unsigned char* dst = base + sw128(32 * k + m, c & 7);
                        if (row != 0xffffffffu) cp_async16(dst, a.q + (size_t)row * D + c * 8);
                        else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
                    }
                cp_async_wait_all();
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full);
            ++it;
        }
        // the tables of a group's requests have to name its first one's pages
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            const int g = a.p.gid[b];
            if (g < 0) continue;
            const Group grp = a.p.group[g];
            const int32_t* mine = a.block_table + (size_t)b * a.max_pages;
            const int32_t* first = a.block_table + (size_t)grp.leader * a.max_pages;
            bool differ = false;
            for (int j = t0; j < grp.positions / a.page_size; j += 64) differ = differ || mine[j] != first[j];
            if (differ) rd_flag(a.status, RD_DEV_BAD_INDEX);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        // The MMAs of one thread run in issue order, so S_t(j + 1) may overwrite
        // P_t(j) right behind PV_t(j), and the commit that completes it also
        // covers PV_t(j): softmax t finds O_t stable when it rescales.
        // The whole warp walks the loop and one elected lane issues: the operands
        // are then the same in all lanes and stay in uniform registers.  With only
        // lane 0 in the loop each of the 32 MMAs of a chunk took the issuer 109
        // cycles, against the 64 that the tensor core needs.  Every elected block ends
        // in __syncwarp: a lane that ran ahead into the next wait could hold up the
        // one that has yet to issue what that wait is for.
        constexpr uint32_t idS = idesc_bf16(kM, kN, false, false);
        constexpr uint32_t idSh = idesc_bf16(kM, kN / 2, false, false);
        constexpr uint32_t idPV = idesc_bf16(kM, D, false, true);
        constexpr uint32_t kStage16 = C::kStageBytes >> 4;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // descriptors: only the low word (the start address) changes
        const uint64_t k_desc = smem_desc(smem_addr(smem), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = smem_desc(smem_addr(smem), kN * 128, 1024, kSwizzle128B);
        const uint64_t q_desc = smem_desc(smem_addr(smem + C::kQOff), 16, 1024, kSwizzle128B);
        const uint32_t k_lo = __shfl_sync(0xffffffffu, (uint32_t)k_desc, 0), k_hi = (uint32_t)(k_desc >> 32);
        const uint32_t v_lo = __shfl_sync(0xffffffffu, (uint32_t)v_desc, 0), v_hi = (uint32_t)(v_desc >> 32);
        const uint32_t q_lo = __shfl_sync(0xffffffffu, (uint32_t)q_desc, 0), q_hi = (uint32_t)(q_desc >> 32);
        const bool leader = elect_one();
        if (a.stall_budget > 0 && !warp_wait(&bar.never, 0, abort, a.stall_budget)) fail();
        uint32_t st = 0, ph = 0;                          // the ring's next entry, its phase
        uint32_t it = 0;                                  // units
        uint32_t pp[2] = {0u, 0u};                        // phase of p_full
        uint32_t ut[2] = {0u, 0u};                        // units with tile t so far
        auto step = [&](uint32_t& s_, uint32_t& p_) {     // take the ring's next entry
            s_ = st;
            p_ = ph;
            if (++st == (uint32_t)C::kStages) {
                st = 0;
                ph ^= 1u;
            }
        };
        auto commit = [&](uint64_t* b) {
            if (leader) mma_commit(b);
            __syncwarp();
        };
        auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(b, parity, abort, kWaitBudget); };
        Walk w;
        w.begin(a);
        Piece u;
        while (!*abort && w.next(a, u)) {
            const int n = __shfl_sync(0xffffffffu, u.n, 0);
            const int nb = __shfl_sync(0xffffffffu, u.rows, 0) > kM ? 2 : 1;      // active tiles
            // an odd last half: 64 positions
            const int odd = __shfl_sync(0xffffffffu, (u.c0 + u.n - 1) * kN + 64 >= u.g.positions ? u.n - 1 : -1, 0);
            auto issue_s = [&](int t, uint32_t ks, int j) {
                const uint32_t id = j == odd ? idSh : idS;
                const uint32_t kd = k_lo + ks * kStage16, qd = q_lo + t * (C::kQBytes >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * (kM * 128) + (k & 3) * 32) >> 4;
                        mma_smem_a(tm + C::s_col(t), desc64(qd + off, q_hi), desc64(kd + off, k_hi), id, k > 0);
                    }
                    mma_commit(&bar.s_full[t]);
                }
                __syncwarp();
            };
            uint32_t ks, kp, vs, vp;
            step(ks, kp);
            bool ok = wait(&bar.q_full, it & 1) && wait(&bar.kv_full[ks], kp);
            if (!ok) { fail(); break; }
            tc_fence_after();
            issue_s(0, ks, 0);
            if (nb == 2) issue_s(1, ks, 0);
            commit(&bar.kv_empty[ks]);
            if (n == 1) commit(&bar.q_free);
            for (int j = 0; ok && j < n; ++j) {
                const bool more = j + 1 < n;
                step(vs, vp);
                if (more) step(ks, kp);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= nb) break;
                    if (t == 0) ok = wait(&bar.kv_full[vs], vp);
                    if (j == 0 && ut[t] > 0) ok = ok && wait(&bar.o_free[t], (ut[t] - 1) & 1);
                    ok = ok && wait(&bar.p_full[t], pp[t]);
                    if (!ok) break;
                    pp[t] ^= 1u;
                    tc_fence_after();
                    const uint32_t vd = v_lo + vs * kStage16;
                    if (leader) {
                        // the weights of the second 64 positions lie 64 columns on
#pragma unroll
                        for (int k = 0; k < kN / 16; ++k)
                            if (k < kN / 32 || j != odd)
                                mma_tmem_a(tm + C::o_col(t), tm + C::s_col(t) + (k >> 2) * 64 + (k & 3) * 8,
                                           desc64(vd + k * 128, v_hi), idPV, j > 0 || k > 0);
                    }
                    __syncwarp();
                    if (t == nb - 1) commit(&bar.kv_empty[vs]);
                    if (more) {
                        if (t == 0) ok = wait(&bar.kv_full[ks], kp);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(t, ks, j + 1);
                        if (t == nb - 1) {
                            commit(&bar.kv_empty[ks]);
                            if (j + 2 == n) commit(&bar.q_free);
                        }
                    } else {
                        commit(&bar.o_final[t]);
                    }
                }
            }
            if (!ok) { fail(); break; }
            ++ut[0];
            if (nb == 2) ++ut[1];
            ++it;
        }
        // drain: every issued MMA must finish before TMEM is freed
        commit(&bar.drain);
        mbar_wait(&bar.drain, 0, &no_abort, kWaitBudget);
    }
    } else {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 3, half = (warp >> 2) & 1;  // tile, half of the chunk's positions
        const int r = tid & (kM - 1);                     // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sc = tmem + lane_base + C::s_col(t) + half * 64;     // this half's scores
        constexpr int DH = D / 2;                         // this thread's columns of O
        const uint32_t oc = tmem + lane_base + C::o_col(t) + half * DH;
        float* const share = reinterpret_cast<float*>(smem + C::kShareOff) + t * kM + r;
        // The eight warps of a tile go through the same barriers whatever happens: a
        // wait that ran out joins the next reduction and all of them leave together.
        auto any_of_tile = [&](bool p) { return barrier_or(1 + t, 256, p); };
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
        uint32_t ct = 0, ut = 0;
        Walk w;
        w.begin(a);
        Piece u;
        while (w.next(a, u)) {
            const int row = t * kM + r;                   // row of the unit
            if (t == 1 && u.rows <= kM) continue;
            const bool valid = row < u.rows;
            // a warp without a valid row leaves S where P belongs: its rows of O are
            // never read
            const bool dead = __all_sync(0xffffffffu, !valid);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < u.n; ++j) {
                ok = warp_wait(&bar.s_full[t], (ct + j) & 1, abort, kWaitBudget);
                tc_fence_after();
                // the odd last chunk has 64 positions: none for the second half
                const bool mine = ok && !dead && (half == 0 || (u.c0 + j) * kN + 64 < u.g.positions);
                uint32_t pv[32];                          // this half's weights, as bf16 pairs
                uint64_t sum[2];
                // Weights against the maximum so far, and the scores' own: only where
                // that has grown too much are they worked out again, from the same
                // scores (nothing is written before the tile has agreed)
                auto weights = [&]() -> float {
                    const float base = m == -INFINITY ? 0.f : m;
                    const uint64_t base2 = pack2(-base, -base);
                    float mx[4];
                    sum[0] = sum[1] = 0ull;
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 16) {
                        uint32_t s[16];
                        tmem_ld16(sc + c0, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float y0 = __uint_as_float(s[2 * e]), y1 = __uint_as_float(s[2 * e + 1]);
                            mx[e & 3] = c0 == 0 && e < 4 ? fmaxf(y0, y1) : fmaxf(fmaxf(mx[e & 3], y0), y1);
                            float x0, x1;
                            unpack2(fma2(pack2(y0, y1), scale2, base2), x0, x1);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                            pv[c0 / 2 + e] = pack_bf16(p0, p1);
                        }
                    }
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                };
                float ms = -INFINITY;
                if (mine) ms = weights();
                if (any_of_tile(!ok || ms > m + kRescaleThreshold)) {
                    if (any_of_tile(!ok)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 32; ++i) pv[i] = 0u;      // (nothing to keep over the exchange)
                    if (half == 1) *share = ms;
                    any_of_tile(false);
                    if (half == 0) {
                        const float top = fmaxf(ms, *share);
                        ms = top > m + kRescaleThreshold ? top : m;
                        *share = ms;
                    }
                    any_of_tile(false);
                    if (half == 1) ms = *share;           // the row's maximum from here on
                    const float f = ms != m ? fast_exp2(m - ms) : 1.f;    // 0 while m is -inf
                    l *= f;
                    m = ms;
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                        for (int cb = 0; cb < DH / 32; ++cb) {
                            uint32_t o[32];
                            tmem_ld32(oc + cb * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            tmem_st32(oc + cb * 32, o);
                        }
                        tmem_st_wait();
                    }
                    if (mine) weights();
                    // (PV adds to all columns of O: it waits for both halves' arrivals below)
                }
                if (mine) {
                    tmem_st32(sc, pv);                    // over this half's scores
                    float a0, a1;
                    unpack2(add2(sum[0], sum[1]), a0, a1);
                    l += a0 + a1;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[t]);
            }
            if (ok) ok = warp_wait(&bar.o_final[t], ut & 1, abort, kWaitBudget);
            else { fail(); break; }                       // (every warp of the tile leaves here)
            if (half == 1) *share = l;
            if (any_of_tile(!ok)) { fail(); break; }
            tc_fence_after();
            // fp32 partials, four columns of consecutive rows side by side
            const bool whole = u.slot < 0;
            const size_t stride = whole ? a.p.rows_cap : kUnitRows;
            const size_t at = whole ? (size_t)u.g.node0 * a.G + u.row0 + row : (size_t)row;
            const size_t block = whole ? u.h : u.slot;
            float4* dst = (whole ? a.p.rows : a.p.part) + (block * (D / 4) + half * (DH / 4)) * stride + at;
#pragma unroll
            for (int cb = 0; cb < DH / 32; ++cb) {
                uint32_t o[32];
                tmem_ld32(oc + cb * 32, o);
                tmem_ld_wait();
                if (cb == DH / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.o_free[t]);
                }
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[(size_t)(cb * 8 + i) * stride] =
                            make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                        __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
            }
            if (valid && half == 0)
                (whole ? a.p.rows_ml : a.p.part_ml)[block * stride + at] = make_float2(m, l + *share);
            ct += u.n;
            ++ut;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ----------------------------------------------------------------------- merge
// CTA = (request, kv head, R rows p G + g).  What bounds it is the chain of reads
// that leads to the partials (request, unit, then (m, l) and O), so each CTA walks
// that chain once for its rows and then has all their pieces on the way at the same
// time: copies into shared memory (cp.async) hold no registers.  A row's pieces are
// those of its prefix unit and of its suffix unit, kMergePieces of them a round.
// Few rows a CTA: many CTAs' chains run side by side, and none waits for a second
// wave (32 rows take 69.7 us for the whole call where 8 take 65.7: 16 requests x 8
// heads x 160 rows, 75 of them live; half the columns a thread cost 2 to 6 us on top).
struct MergeArgs {
    int P_max, Hq, Hkv, G, B;
    int blocks;               // CTAs per (request, kv head)
    bool table;               // suffix units have an entry in the table of pieces
    Plan p;
    uint16_t* o;
};
constexpr int kMergeQ = 4;                 // float4 columns of a thread
constexpr int kMergePieces = 4;
constexpr int kMergeRows = 8;
template <int D> constexpr int kMergeThreads = kMergeRows * (D / 4 / kMergeQ);
template <int D> constexpr int kMergeSmem = kMergePieces * kMergeRows * D * 4;

template <int D>
__global__ void __launch_bounds__(kMergeThreads<D>)
merge_kernel(const MergeArgs a)
{
    extern __shared__ float4 stage[];                     // [piece][D / 4][kMergeRows]
    __shared__ Pieces s_pc[2][kMergeRows];
    constexpr int kQ = kMergeQ, kParts = D / 4 / kQ;      // threads of a row
    const int bh = blockIdx.x / a.blocks;
    const int b = bh / a.Hkv, h = bh % a.Hkv;
    const int row0 = (blockIdx.x % a.blocks) * kMergeRows;
    const int tid = threadIdx.x;
    const int r = tid % kMergeRows, part = tid / kMergeRows, row = row0 + r;      // row = p G + g
    const int all = a.P_max * a.G;
    // the plan is written: the suffix kernel's launch has waited for it
    const int len = __ldcg(a.p.eff_len + b);
    const int4 req = __ldcg(a.p.req + b);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int n = 0;                                            // the row's pieces
    if (part == 0 && row < all) {
        int2 su = make_int2(1, 0);                        // (a skipped request's entry is not used)
        if (a.table) su = __ldcg(a.p.suffix.unit + ((size_t)(row / a.p.slot_rows) * a.B + b) * a.Hkv + h);
        Pieces pre = {};
        const bool in = row < len * a.G;
        if (in && req.x >= 0) {
            const int gr = req.z + row;
            pre = pieces_of<D>(__ldcg(a.p.unit + req.x + h * req.y + gr / kUnitRows), a.p, h, req.w + row,
                               gr % kUnitRows);
        }
        s_pc[0][r] = pre;
        s_pc[1][r] = pieces_at<D>(su, a.p.suffix.rows, a.p.suffix.rows_ml, a.p.suffix.rows_cap, h, (size_t)b * all + row,
                                  a.p.suf_part, a.p.suf_part_ml, a.p.slot_rows, row % a.p.slot_rows, a.p.suf_grid);
        n = in ? pre.n + s_pc[1][r].n : 0;
    }
    const int live = min(kMergeRows, len * a.G - row0);   // may be <= 0
    int most = n;                                         // of the CTA's rows
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    __shared__ int s_most[kMergeThreads<D> / 32];
    if ((tid & 31) == 0) s_most[tid >> 5] = most;
    __syncthreads();
    most = 0;
#pragma unroll
    for (int i = 0; i < kMergeThreads<D> / 32; ++i) most = max(most, s_most[i]);
    n = r < live ? s_pc[0][r].n + s_pc[1][r].n : 0;
    float M = -INFINITY, L = 0.f;
    float4 acc[kQ];
#pragma unroll
    for (int e = 0; e < kQ; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < most; k0 += kMergePieces) {
        // the round's pieces: thread part of row r fetches its own columns
        float2 ml[kMergePieces];
#pragma unroll
        for (int i = 0; i < kMergePieces; ++i) {
            const int k = k0 + i;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (k < n) {
                const int pn = s_pc[0][r].n;
                const Pieces& q = s_pc[k < pn ? 0 : 1][r];
                const int kk = k < pn ? k : k - pn;
                const float4* src = q.o(kk) + (size_t)(part * kQ) * q.stride;
                const size_t stride = q.stride;
#pragma unroll
                for (int e = 0; e < kQ; ++e)
                    cp_async16(stage + (i * (D / 4) + part * kQ + e) * kMergeRows + r, src + (size_t)e * stride);
                ml[i] = __ldcg(q.ml(kk));
            }
        }
        cp_async_wait_all();                              // each thread reads only what it fetched
        float Mn = M;
#pragma unroll
        for (int i = 0; i < kMergePieces; ++i) Mn = fmaxf(Mn, ml[i].x);
        const float base = Mn == -INFINITY ? 0.f : Mn;    // no visible key yet (or only NaN scores)
        const float keep = exp2f(M - base);               // 0 while M is -inf
        M = Mn;
        L *= keep;
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
            acc[e].x *= keep; acc[e].y *= keep; acc[e].z *= keep; acc[e].w *= keep;
        }
#pragma unroll
        for (int i = 0; i < kMergePieces; ++i) {
            if (k0 + i >= n) continue;
            const float w = exp2f(ml[i].x - base);
            L += ml[i].y * w;                             // (NaN scores: l = NaN, m = -inf, 0 x NaN)
#pragma unroll
            for (int e = 0; e < kQ; ++e) {
                const float4 x = stage[(i * (D / 4) + part * kQ + e) * kMergeRows + r];
                acc[e].x += x.x * w; acc[e].y += x.y * w; acc[e].z += x.z * w; acc[e].w += x.w * w;
            }
        }
    }
    if (row >= all) return;
    const float inv = r < live ? (L == 0.f ? 0.f : 1.f / L) : 0.f;    // padded rows: zeros
    uint4* dst = reinterpret_cast<uint4*>(
        a.o + (((size_t)b * a.P_max + row / a.G) * a.Hq + h * a.G + row % a.G) * D + part * (D / kParts));
#pragma unroll
    for (int e = 0; e < kQ; e += 2)
        dst[e / 2] = make_uint4(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv),
                                pack_bf16(acc[e + 1].x * inv, acc[e + 1].y * inv),
                                pack_bf16(acc[e + 1].z * inv, acc[e + 1].w * inv));
}

// ------------------------------------------------------------------ host side
template <int D>
cudaError_t launch_merge(dim3 grid, cudaStream_t stream, MergeArgs& a)
{
    cudaError_t e = cudaFuncSetAttribute(merge_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMergeSmem<D>);
    if (e != cudaSuccess) return e;
    void* args[] = {&a};
    return launch_dependent(reinterpret_cast<const void*>(merge_kernel<D>), grid, dim3(kMergeThreads<D>), kMergeSmem<D>,
                            stream, args);
}

// Which kernel takes the part behind the prefix.  Up to 128 rows per kv head (and 64
// nodes) the one of shared_suffix.cu, in units of up to 64 rows that read each key
// once; with more the tcgen05 kernel, whose tiles hold 128.  The whole call, 64
// requests of 8 kv heads behind 2,048 shared positions, either way (rows as allocated,
// P_max G; about half of them live): 96 rows and up to 300 positions each 70 against 88
// us, up to 4,000 169 against 180; but 160 rows and up to 3,000 positions 283 against 185
// (to 300: 84 against 102).  16 requests of 80 rows, D 64, to 3,000: 52 against 63; four
// of 128 rows, to 8,000: 44 against 43.
constexpr int kSuffixMaxRows = 128;
constexpr int kSuffixMaxNodes = 64;        // (two mask words a row)
struct SuffixChoice {
    bool few_rows;
    bool by_unit;             // few_rows: CTAs take whole units off a counter and write the output
    bool table;               // units have an entry in the table of pieces
    int grid, slot_rows, tiles;   // tiles: units of a (request, kv head)
    int nodes;                // few_rows: of a unit
    rd_attn_plan plan;        // tcgen05
};
SuffixChoice choose_suffix(int B, int P_max, int Hq, int Hkv, int D, int max_ctx)
{
    SuffixChoice s;
    const int G = Hq / Hkv;
    s.few_rows = P_max <= kSuffixMaxNodes && G <= kSuffixRows && P_max * G <= kSuffixMaxRows;
    s.nodes = s.few_rows ? rd_suffix_nodes(P_max, G) : P_max;
    const int rows = s.nodes * G;
    s.plan = rd_attn_make_plan(B, P_max, Hq, Hkv, D, max_ctx);
    s.grid = s.few_rows ? rd_suffix_grid(rows) : s.plan.grid;
    s.tiles = s.few_rows ? (P_max + s.nodes - 1) / s.nodes : s.plan.tiles;
    s.by_unit = s.few_rows && rd_suffix_by_unit((long long)B * Hkv * s.tiles, s.grid);
    s.table = s.few_rows ? !s.by_unit : s.plan.stream_k;
    s.slot_rows = s.few_rows ? rows : kM;
    return s;
}

// Workspace layout; `base` null: the size only.  The suffix's own workspace (its
// slots, as rd_attn_make_plan sizes them) comes last.
size_t layout(Plan& p, void*& suffix_ws, unsigned char* base, int B, int P_max, int Hq, int Hkv, int D,
              int n_groups, int pre_grid, const SuffixChoice& suffix)
{
    size_t at = 0;
    auto take = [&](auto*& ptr, size_t n) {
        using T = std::remove_reference_t<decltype(*ptr)>;
        ptr = base == nullptr ? nullptr : reinterpret_cast<T*>(base + at);
        at += (n * sizeof(T) + 255) & ~size_t(255);
    };
    p.rows_cap = (size_t)B * P_max * (Hq / Hkv);
    const size_t slots = (size_t)2 * pre_grid;
    take(p.eff_len, B);
    take(p.skip, B);
    take(p.gid, B);
    take(p.node_base, (size_t)B + 1);
    take(p.node_row, (size_t)B * P_max);
    take(p.group, n_groups);
    take(p.first, (size_t)n_groups + 1);
    take(p.req, B);
    take(p.unit, (p.rows_cap / kUnitRows + n_groups) * Hkv);
    take(p.rows, p.rows_cap * Hkv * (D / 4));
    take(p.rows_ml, p.rows_cap * Hkv);
    take(p.part, slots * kUnitRows * (D / 4));
    take(p.part_ml, slots * kUnitRows);
    take(p.suffix.rows, suffix.by_unit ? 0 : p.rows_cap * Hkv * (D / 4));
    take(p.suffix.rows_ml, suffix.by_unit ? 0 : p.rows_cap * Hkv);
    take(p.suffix.unit, suffix.table ? (size_t)suffix.tiles * B * Hkv : 0);
    take(p.suf_first, suffix.few_rows ? (size_t)B + 1 : 0);
    take(p.suf_next, 1);
    p.suffix.rows_cap = p.rows_cap;
    p.suffix.skip = p.skip;
    p.slot_rows = suffix.slot_rows;
    p.grid = pre_grid;
    p.suf_grid = suffix.grid;
    suffix_ws = base == nullptr ? nullptr : base + at;
    const size_t suf_rows = suffix.by_unit ? 0 : (size_t)2 * suffix.grid * suffix.slot_rows;
    p.suf_part = static_cast<float4*>(suffix_ws);
    p.suf_part_ml = reinterpret_cast<float2*>(p.suf_part + suf_rows * (D / 4));
    return at + (suffix.few_rows ? suf_rows * (D * sizeof(float) + sizeof(float2)) : suffix.plan.ws_bytes);
}

template <int D>
cudaError_t launch_prefix(int grid, cudaStream_t stream, PrefixArgs& a, CUtensorMap& mk, CUtensorMap& mv)
{
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    void* args[] = {&a, &mk, &mv};
    return launch_dependent(reinterpret_cast<const void*>(prefix_kernel<D>), dim3(grid), dim3(kThreads),
                            Cfg<D>::kSmemBytes, stream, args);
}

}  // namespace

bool rd_shared_suffix_counts(int B, int P_max, int Hq, int Hkv, int D, int max_ctx)
{
    const SuffixChoice s = choose_suffix(B, P_max, Hq, Hkv, D, max_ctx);
    // units (and twice as many numbers as CTAs drawn behind the last off the counter)
    long long n = (long long)B * Hkv * s.tiles;
    if (s.few_rows && !s.by_unit) {
        // divided into ranges: all chunks, those of the context and of the drafts rounded up
        const int ch = rd_suffix_chunk(rd_suffix_row_warps(s.nodes * (Hq / Hkv)));
        n *= max_ctx / ch + 1LL + P_max / ch + 1LL;
    }
    return n <= 0x7fffffffLL - 4LL * s.grid;              // (the tcgen05 kernel counts chunks only where they fit)
}

size_t rd_shared_workspace_bytes(int B, int P_max, int Hq, int Hkv, int D, int max_ctx, int n_groups)
{
    Plan p;
    void* suffix_ws;
    return layout(p, suffix_ws, nullptr, B, P_max, Hq, Hkv, D, n_groups, rd_device_sm_count(),
                  choose_suffix(B, P_max, Hq, Hkv, D, max_ctx));
}

cudaError_t rd_launch_shared_attention(int B, int P_max, int Hq, int Hkv, int D, float scale, const void* q,
                                       const void* k_new, const void* v_new, const void* k_pool,
                                       const void* v_pool, const rd_paged_kv& paged, int max_ctx,
                                       int n_groups, const int32_t* group_offsets,
                                       const int32_t* prefix_pages, const int32_t* packed_len,
                                       const uint32_t* mask, int mask_words, void* o, void* workspace,
                                       int32_t* dev_status, cudaStream_t stream)
{
    const SuffixChoice suffix = choose_suffix(B, P_max, Hq, Hkv, D, max_ctx);
    const int pre_grid = rd_device_sm_count();
    PlanArgs pa = {};
    pa.B = B;
    pa.P_max = P_max;
    pa.Hkv = Hkv;
    pa.G = Hq / Hkv;
    pa.page_size = paged.page_size;
    pa.max_pages = paged.max_pages;
    pa.max_ctx = max_ctx;
    pa.n_groups = n_groups;
    pa.suffix_chunk = suffix.few_rows && !suffix.by_unit ? rd_suffix_chunk(rd_suffix_row_warps(suffix.nodes * pa.G)) : 0;
    pa.suffix_nodes = suffix.nodes;
    pa.lens = packed_len;
    pa.ctx_lens = paged.ctx_lens;
    pa.group_offsets = group_offsets;
    pa.prefix_pages = prefix_pages;
    pa.status = dev_status;
    void* suffix_ws;
    layout(pa.p, suffix_ws, static_cast<unsigned char*>(workspace), B, P_max, Hq, Hkv, D, n_groups, pre_grid, suffix);
    if (B <= kScanThreads && n_groups <= kScanThreads) plan_kernel<true><<<1, kScanThreads, 0, stream>>>(pa);
    else plan_kernel<false><<<1, kScanThreads, 0, stream>>>(pa);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    PrefixArgs fa = {};
    fa.B = B;
    fa.Hq = Hq;
    fa.Hkv = Hkv;
    fa.G = pa.G;
    fa.page_size = paged.page_size;
    fa.max_pages = paged.max_pages;
    fa.num_pages = paged.num_pages;
    fa.n_groups = n_groups;
    fa.scale_log2 = scale * kLog2e;
    fa.q = static_cast<const uint16_t*>(q);
    fa.block_table = paged.block_table;
    fa.p = pa.p;
    fa.status = dev_status;
    fa.stall_budget = rd_attention_stall_budget();
    CUtensorMap mk, mv;
    const int64_t pool_rows = (int64_t)paged.num_pages * paged.page_size;
    if (!make_kv_map(&mk, k_pool, pool_rows, Hkv, D) || !make_kv_map(&mv, v_pool, pool_rows, Hkv, D))
        return cudaErrorInvalidValue;
    e = D == 128 ? launch_prefix<128>(pre_grid, stream, fa, mk, mv) : launch_prefix<64>(pre_grid, stream, fa, mk, mv);
    if (e != cudaSuccess) return e;

    if (suffix.few_rows)
        e = rd_launch_shared_suffix(pa.p, B, P_max, Hq, Hkv, D, fa.scale_log2, q, k_new, v_new, k_pool, v_pool, paged,
                                    mask, mask_words, suffix.by_unit, o, dev_status, stream);
    else
        e = rd_launch_attention(suffix.plan, B, P_max, Hq, Hkv, D, scale, q, k_new, v_new, k_pool, v_pool, nullptr, 0, max_ctx,
                                pa.p.eff_len, mask, mask_words, o, suffix_ws, dev_status, stream, &paged, nullptr,
                                &pa.p.suffix);
    if (e != cudaSuccess || suffix.by_unit) return e;      // (its units end in output rows)

    MergeArgs ma = {};
    ma.P_max = P_max;
    ma.Hq = Hq;
    ma.Hkv = Hkv;
    ma.G = pa.G;
    ma.B = B;
    ma.blocks = (P_max * pa.G + kMergeRows - 1) / kMergeRows;
    ma.table = suffix.table;
    ma.p = pa.p;
    ma.o = static_cast<uint16_t*>(o);
    const dim3 merge_grid((unsigned)((size_t)B * Hkv * ma.blocks));
    return D == 128 ? launch_merge<128>(merge_grid, stream, ma) : launch_merge<64>(merge_grid, stream, ma);
}
