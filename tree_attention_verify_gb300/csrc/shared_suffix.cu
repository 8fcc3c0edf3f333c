// The part of rd_tree_attention_shared behind the prefix, for up to 128 query rows
// per kv head (P_max G): fp32 partials of every live row over its request's own
// context and its drafts.
//
// Unit = (request, kv head, up to 64 rows: as many nodes, with all their G heads, as
// fit).  Behind a shared prompt a request has a few hundred positions of its own, so a
// unit is a handful of chunks, and what bounds it is not bytes or products but the chain of steps per unit.  The tcgen05 kernel pays that chain
// across four roles (64 positions take it 2,500 to 4,000 cycles behind a prefix, its
// epilogue 4,000 more): 120 us at 64 requests x 40 heads x 150 positions and 23 live
// rows of 48.  Here a warp holds 16 rows' queries, scores, statistics and sums in its own
// registers (mma.sync m16n8k16), so that nothing waits on another role but for
// loads, and two or three CTAs share an SM.  With 64 rows or fewer the products stay
// under what mma.sync can do at the rate the keys arrive.
//
// Warp roles: one producer (TMA: a unit's queries and what the others need to know
// of it, then its chunks of CH positions through a ring of ST stages), NW x KS
// compute warps: NW of 16 rows each, times KS that split each chunk's positions
// (few rows) and join their sums in shared memory at the unit's end.  With many
// units the CTAs take them whole off a counter, as they come free from the prefix
// (equal ranges, begun when the prefix's CTAs end, left the last one 35 us behind the
// median at 2,560 units).  Each unit then ends with its rows' partials over the
// prefix, which come through the same ring like further chunks, and with the output
// rows: no partials of its own leave the SM, and no merge follows.  At 64 requests x
// 40 heads that takes 73 us (355 MB from and to HBM, 4.9 TB/s) where this kernel and
// the merge took 48 + 36.  With few units, their chunks form one sequence that the
// CTAs take in equal ranges, and all partials go to the merge.
// Every wait is bounded; on expiry the CTA records RD_DEV_TIMEOUT, drains its
// copies and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "rd_internal.cuh"
#include "shared_prefix.cuh"
#include "tc_ptx.cuh"

namespace {
using namespace rdtc;
using namespace rdattn;
using namespace rdshared;

constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when a maximum grows by > 2^8
constexpr long long kWaitBudget = 4000000000LL;   // ~2 s of SM clock per wait

template <int D, int NW, int KS> struct SCfg {
    static constexpr int kCh = rd_suffix_chunk(NW);     // positions of a chunk
    static constexpr int kKw = kCh / KS;                // positions of a warp in a chunk
    static constexpr int kStages = NW <= 2 ? 2 : NW == 3 ? 3 : 4;
    static constexpr int kWarps = NW * KS;
    static constexpr int kThreads = (kWarps + 1) * 32;
    static constexpr int kDB = D / 64;
    static constexpr int kKBytes = kCh * D * 2;
    static constexpr int kStageBytes = 2 * kKBytes;
    static constexpr int kQRows = NW * 16;
    static constexpr int kQBytes = kQRows * D * 2;
    static constexpr int kQOff = kStages * kStageBytes;
    static constexpr int kJoinOff = kQOff + kQBytes;                // (KS - 1) NW warps' sums
    static constexpr int kJoinBytes = (KS - 1) * NW * (16 * D * 4 + 16 * 8);
    static constexpr int kMlOff = kJoinOff + kJoinBytes;            // (m, l) of a stage's rows over the prefix
    static constexpr int kMlRows = kQRows + 2;
    static constexpr int kBarOff = kMlOff + kStages * kMlRows * 8;
    static constexpr int kSmemBytes = kBarOff + 512 + 1024;
    static constexpr int kCtas = rd_suffix_ctas(NW);                // per SM
    static_assert(kCtas * (kSmemBytes + 1024) <= 227 * 1024, "CTAs per SM");
    static_assert(kKw % 16 == 0, "a warp's positions are whole k-steps");
    // half the columns of every row's partials fit a stage
    static_assert(kQRows * (D / 2) * 4 <= kStageBytes, "partials in the ring");
    static_assert(kMlOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

struct SuffixArgs {
    int B, P_max, Hq, Hkv, G, page_size, max_pages, num_pages, mask_words;
    int nodes, blocks;         // of a unit at most; units of a (request, kv head)
    float scale_log2;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    const uint32_t* mask;
    uint16_t* o;
    Plan p;
    bool by_unit;
    int32_t* status;
    long long stall_budget;
};

// What the compute warps need to know of a unit (or piece); n = 0: no more, -1: a
// skipped request's rows (zeros).
struct Unit {
    int row0, h;               // first node b P_max + n0
    int rows;                  // live rows, and << 16 those with padded nodes
    int n, C, Pb, slot;        // Pb: the request's nodes; slot -1: a whole unit
};

// What a ring entry holds.
struct Entry {
    int kind;                              // 0: chunk c of the unit, 1: partials over the prefix, 2: nothing
    int c, last;                           // last: the unit ends with it
    int r0, r1, half, shift;               // partials: rows [r0, r1), half of the columns; first (m, l) at `shift`
};

struct SBar {
    uint64_t full[4];
    uint64_t empty[4];
    uint64_t q_full;       // a unit's queries, and `unit`
    uint64_t q_empty;      // every compute warp has both in registers
    uint64_t join_full;
    uint64_t join_empty;
    uint64_t never;
    Unit unit;
    Entry entry[4];
    int abort;
};
static_assert(sizeof(SBar) <= 512, "barrier block");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four lanes with four words each: word k of lane t becomes word t of lane k.
__device__ __forceinline__ void swap4(uint32_t (&v)[4], int t)
{
    const bool odd = t & 1, high = t & 2;
    const uint32_t a0 = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
    const uint32_t a1 = __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[3], 1);
    if (odd) { v[0] = a0; v[2] = a1; } else { v[1] = a0; v[3] = a1; }
    const uint32_t b0 = __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 2);
    const uint32_t b1 = __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 2);
    if (high) { v[0] = b0; v[1] = b1; } else { v[2] = b0; v[3] = b1; }
}

template <int D, int NW, int KS>
__global__ void __launch_bounds__((NW * KS + 1) * 32, SCfg<D, NW, KS>::kCtas)
suffix_kernel(const SuffixArgs a, const __grid_constant__ CUtensorMap map_kc,
              const __grid_constant__ CUtensorMap map_vc, const __grid_constant__ CUtensorMap map_kd,
              const __grid_constant__ CUtensorMap map_vd, const __grid_constant__ CUtensorMap map_q,
              const __grid_constant__ CUtensorMap map_rows, const __grid_constant__ CUtensorMap map_part)
{
    using C = SCfg<D, NW, KS>;
    constexpr int CH = C::kCh;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SBar& bar = *reinterpret_cast<SBar*>(smem + C::kBarOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bar.abort;
    volatile int no_abort = 0;
    // the merge may start now: it waits for this grid before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], C::kWarps);
        }
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, C::kWarps);
        mbar_init(&bar.join_full, (KS - 1) * NW > 0 ? (KS - 1) * NW : 1);
        mbar_init(&bar.join_empty, NW);
        mbar_init(&bar.never, 1);
        bar.abort = 0;
        mbar_fence_init();
    }
    __syncthreads();
    auto fail = [&]() {
        *abort = 1;
        rd_flag(a.status, RD_DEV_TIMEOUT);
    };

    if (warp == C::kWarps) {
        // ------------------------------------------------------------ producer
        const uint32_t W = a.by_unit ? 0u : __ldcg(a.p.suf_first + a.B);
        const uint32_t nc = W > 0u ? range_ctas(W, gridDim.x, kSuffixMinChunks) : 0u;
        uint32_t x = 0u, end = 0u;
        int b = 0;
        uint32_t base = 0u;                               // suf_first[b]
        if (blockIdx.x < nc) {
            x = range_start(W, nc, blockIdx.x);
            end = range_start(W, nc, blockIdx.x + 1);
            // the last request with suf_first <= x, 32 probes at a time
            int lo = 0, hi = a.B;
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32;
                const int at = lo + lane * step;
                const bool le = at < hi && __ldcg(a.p.suf_first + at) <= x;
                const int k = 31 - __clz((int)__ballot_sync(0xffffffffu, le));
                lo += k * step;
                hi = min(hi, lo + step);
            }
            b = lo;
            base = __ldcg(a.p.suf_first + b);
        }
        const uint32_t start = x;
        if (lane == 0) {
            tma_prefetch_desc(&map_kc);
            tma_prefetch_desc(&map_vc);
            tma_prefetch_desc(&map_kd);
            tma_prefetch_desc(&map_vd);
            tma_prefetch_desc(&map_q);
            if (a.by_unit) {
                tma_prefetch_desc(&map_rows);
                tma_prefetch_desc(&map_part);
            }
            if (a.stall_budget > 0 && !mbar_wait(&bar.never, 0, abort, a.stall_budget)) fail();
            uint32_t g = 0, it = 0;
            bool ok = true;
            int len = 0, ctx = 0, skip = 0;               // of request b
            auto request = [&]() {
                len = __ldcg(a.p.eff_len + b);
                skip = __ldcg(a.p.skip + b);
                ctx = __ldg(a.ctx_lens + b) - skip;
            };
            // ranges: the next request's first chunk, chunks of a unit, units of a kv head
            uint32_t next = 0u, nb = 0u, live = 1u;
            bool fresh = true, prefix_written = false;
            // by unit: what is read of a unit comes a unit ahead, its number two ahead
            const int per = a.Hkv * a.blocks, units = a.B * per;
            int unit = units, after = units, n_len = 0, n_ctx_len = 0, n_skip = 0;
            int4 n_req = make_int4(-1, 0, 0, 0);
            auto read_ahead = [&]() {
                if (unit >= units) return;
                const int q = unit / per;
                n_len = __ldcg(a.p.eff_len + q);
                n_skip = __ldcg(a.p.skip + q);
                n_ctx_len = __ldg(a.ctx_lens + q);
                n_req = __ldcg(a.p.req + q);
            };
            if (a.by_unit) {
                unit = atomicAdd(a.p.suf_next, 1);
                after = atomicAdd(a.p.suf_next, 1);
                read_ahead();
            }
            while (ok && !*abort) {
                int h = 0, n0 = 0, c0 = 0, n = 0, slot = -1;
                uint32_t stop = 0u;
                int4 req = make_int4(-1, 0, 0, 0);
                if (a.by_unit) {
                    if (unit < units) {
                        b = unit / per;
                        h = unit % per / a.blocks;
                        n0 = unit % a.blocks * a.nodes;
                        len = n_len;
                        skip = n_skip;
                        ctx = n_ctx_len - skip;
                        req = n_req;
                        unit = after;
                        if (after < units) after = atomicAdd(a.p.suf_next, 1);
                        read_ahead();
                        n = len > n0 ? (ctx + CH - 1) / CH + (len + CH - 1) / CH : -1;
                    }
                } else if (x < end) {
                    while (fresh || x >= next) {          // on to the request that holds chunk x
                        if (!fresh) {
                            ++b;
                            base = next;
                        }
                        fresh = false;
                        next = __ldcg(a.p.suf_first + b + 1);
                        request();
                        live = max(1u, (uint32_t)((len + a.nodes - 1) / a.nodes));
                        nb = (next - base) / ((uint32_t)a.Hkv * live);
                    }
                    const uint32_t at = (x - base) / nb, u0 = base + at * nb;
                    h = (int)(at / live);
                    const int blk = (int)(at % live);
                    n0 = blk * a.nodes;
                    c0 = (int)(x - u0);
                    stop = min(u0 + nb, end);
                    n = (int)(stop - x);
                    slot = (uint32_t)n == nb ? -1 : 2 * (int)blockIdx.x + (c0 == 0 && u0 > start ? 1 : 0);
                    if (c0 == 0)                          // the unit starts here: name its pieces
                        a.p.suffix.unit[(blk * a.B + b) * a.Hkv + h] =
                            make_int2(slot < 0 ? 1 : (int)(range_of(W, nc, u0 + nb - 1) - blockIdx.x) + 1, slot);
                }
                if (it > 0 && !mbar_wait(&bar.q_empty, (it - 1) & 1, abort, kWaitBudget)) { ok = false; break; }
                if (n == 0) {                             // no more
                    bar.unit.n = 0;
                    mbar_arrive(&bar.q_full);
                    break;
                }
                const int live_rows = max(0, min(len - n0, a.nodes)) * a.G;
                bar.unit = Unit{b * a.P_max + n0, h, live_rows | min(a.P_max - n0, a.nodes) * a.G << 16, n, ctx, len, slot};
                if (n < 0) {
                    mbar_arrive(&bar.q_full);
                    ++it;
                    continue;
                }
                mbar_arrive_expect_tx(&bar.q_full, a.nodes * a.G * D * 2);
#pragma unroll
                for (int db = 0; db < C::kDB; ++db)
                    tma_load_3d(smem + C::kQOff + db * (C::kQRows * 128), &map_q, &bar.q_full, db * 64, h * a.G,
                                b * a.P_max + n0);
                ++it;
                // the next ring entry, free; false: the wait ran out
                auto stage = [&](int& st) -> bool {
                    st = (int)(g % C::kStages);
                    return g < (uint32_t)C::kStages ||
                           mbar_wait(&bar.empty[st], ((g / C::kStages) - 1) & 1, abort, kWaitBudget);
                };
                const int n_ctx = (ctx + CH - 1) / CH;
                int entry = -1, page = 0;
                for (int c = c0; c < c0 + n; ++c, ++g) {
                    const CUtensorMap* mk = &map_kd;
                    const CUtensorMap* mv = &map_vd;
                    int z = b * a.P_max + (c - n_ctx) * CH;
                    if (c < n_ctx) {
                        const int pos = skip + c * CH;
                        if (pos / a.page_size != entry) { // one lookup a page
                            entry = pos / a.page_size;
                            page = __ldg(a.block_table + (size_t)b * a.max_pages + entry);
                            if (page < 0 || page >= a.num_pages) {
                                rd_flag(a.status, RD_DEV_BAD_INDEX);
                                page = 0;
                            }
                        }
                        mk = &map_kc;
                        mv = &map_vc;
                        z = page * a.page_size + pos % a.page_size;
                    }
                    int st;
                    if (!stage(st)) { ok = false; break; }
                    unsigned char* ks = smem + st * C::kStageBytes;
                    bar.entry[st] = Entry{0, c, c + 1 == c0 + n && req.x < 0, 0, 0, 0, 0};
                    mbar_arrive_expect_tx(&bar.full[st], C::kStageBytes);
#pragma unroll
                    for (int db = 0; db < C::kDB; ++db) {
                        tma_load_3d(ks + db * (CH * 128), mk, &bar.full[st], db * 64, h, z);
                        tma_load_3d(ks + C::kKBytes + db * (CH * 128), mv, &bar.full[st], db * 64, h, z);
                    }
                }
                x = stop;
                if (!ok || req.x < 0) continue;
                // the rows' partials over the prefix: their unit's pieces (of two units,
                // where the rows cross one's end), half of the columns at a time
                if (!prefix_written) asm volatile("griddepcontrol.wait;" ::: "memory");
                prefix_written = true;
                for (int r0 = 0; ok && r0 < live_rows;) {
                    const int at = req.z + n0 * a.G + r0, r = at % kUnitRows, r1 = min(live_rows, r0 + kUnitRows - r);
                    const int2 table = __ldcg(a.p.unit + req.x + h * req.y + at / kUnitRows);
                    const int pieces = pieces_in(table, a.p.grid);
                    const bool whole = pieces == 1;
                    const int row = req.w + n0 * a.G + r0;                         // compact
                    for (int k = 0; ok && k < pieces; ++k) {
                        const int sl = k == 0 ? table.y : 2 * (table.y / 2 + k);       // its slot
                        const CUtensorMap* map = whole ? &map_rows : &map_part;
                        const int px = (whole ? row : r) * 4, py = (whole ? h : sl) * (D / 4);
                        const float2* ml = whole ? a.p.rows_ml + (size_t)h * a.p.rows_cap + row
                                                 : a.p.part_ml + (size_t)sl * kUnitRows + r;
                        const int shift = (int)((reinterpret_cast<uintptr_t>(ml) >> 3) & 1);   // copies begin at 16 bytes
                        const uint32_t ml_bytes = (uint32_t)((r1 - r0 + shift + 1) & ~1) * 8u;
                        for (int half = 0; half < 2; ++half, ++g) {
                            int st;
                            if (!stage(st)) { ok = false; break; }
                            bar.entry[st] = Entry{1, 0, 0, r0, r1, half, shift};
                            mbar_arrive_expect_tx(&bar.full[st], C::kQRows * 16 * (D / 8) + (half == 0 ? ml_bytes : 0u));
                            tma_load_2d(smem + st * C::kStageBytes, map, &bar.full[st], px, py + half * (D / 8));
                            if (half == 0)
                                bulk_load(smem + C::kMlOff + st * C::kMlRows * 8, ml - shift, ml_bytes, &bar.full[st]);
                        }
                    }
                    r0 = r1;
                }
                int st;
                if (!ok || !stage(st)) { ok = false; continue; }
                bar.entry[st] = Entry{2, 0, 1, 0, 0, 0, 0};
                mbar_arrive(&bar.full[st]);
                ++g;
            }
            if (!ok || *abort) {
                // the compute warps may have left before the last queries landed
                fail();
                if (it > 0) mbar_wait(&bar.q_full, (it - 1) & 1, &no_abort, kWaitBudget);
            }
            // drain: every issued copy must land before the CTA may exit
            for (uint32_t k = g > (uint32_t)C::kStages ? g - C::kStages : 0u; k < g; ++k)
                mbar_wait(&bar.full[k % C::kStages], (k / C::kStages) & 1, &no_abort, kWaitBudget);
        }
    } else {
        // ------------------------------------------------------------- compute
        const int rw = warp % NW, ks = warp / NW;         // 16 rows, share of a chunk's positions
        const int gr = lane >> 2, tc = lane & 3;
        const uint32_t smem_u = smem_addr(smem);
        // ldmatrix rows of this lane: queries (A), keys (B, two tiles of 8), values (B, transposed)
        const int a_row = rw * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, a_c = lane >> 4;
        const int k_row = ks * C::kKw + (lane & 7) + ((lane >> 4) & 1) * 8, k_c = (lane >> 3) & 1;
        const int v_row = ks * C::kKw + (lane & 7) + ((lane >> 3) & 1) * 8, v_c = lane >> 4;
        uint32_t g = 0, it = 0, joins = 0;
        bool ok = true;
        for (;; ++it) {
            if (!warp_wait(&bar.q_full, it & 1, abort, kWaitBudget)) { ok = false; break; }
            const Unit u = bar.unit;
            if (u.n == 0) break;
            const int live = u.rows & 0xffff;             // rows of the unit
            const bool dead = rw * 16 >= live;            // none of this warp's
            uint32_t qf[D / 16][4];
            if (!dead) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    ldsm4(qf[k], smem_u + C::kQOff + (k >> 2) * (C::kQRows * 128) +
                                     sw128(a_row, (k & 3) * 2 + a_c));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_empty);
            // ancestor bits of this thread's two rows (drafts 0-31, 32-63)
            uint32_t mw[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = rw * 16 + gr + 8 * i;
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    mw[i][w] = row < live && w < a.mask_words
                        ? __ldg(a.mask + (size_t)(u.row0 + row / a.G) * a.mask_words + w) : 0u;
            }
            float o[D / 8][4];
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            float wp[2] = {0.f, 0.f};                     // weights of the prefix piece at hand
            // the unit's own sums: over a row's four lanes, then over the warps that split
            // the positions (those of ks > 0 leave theirs and only keep step from there on)
            auto finish = [&]() -> bool {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                }
                if constexpr (KS > 1) {
                    float* const jo = reinterpret_cast<float*>(smem + C::kJoinOff);
                    float2* const jml = reinterpret_cast<float2*>(smem + C::kJoinOff + (KS - 1) * NW * 16 * D * 4);
                    if (ks > 0) {
                        if (joins > 0 && !warp_wait(&bar.join_empty, (joins - 1) & 1, abort, kWaitBudget)) return false;
                        ++joins;
                        const int at = (ks - 1) * NW + rw;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j)
                            *reinterpret_cast<float4*>(jo + ((size_t)(at * (D / 8) + j) * 32 + lane) * 4) =
                                make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
                        if (tc == 0) {
                            jml[at * 16 + gr] = make_float2(m[0], l[0]);
                            jml[at * 16 + gr + 8] = make_float2(m[1], l[1]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.join_full);
                        return true;
                    }
                    if (!warp_wait(&bar.join_full, joins & 1, abort, kWaitBudget)) return false;
                    ++joins;
#pragma unroll
                    for (int t = 0; t < KS - 1; ++t) {
                        const int at = t * NW + rw;
                        float f[2], q[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 ml = jml[at * 16 + gr + 8 * i];
                            const float M = fmaxf(m[i], ml.x), base = M == -INFINITY ? 0.f : M;
                            f[i] = fast_exp2(m[i] - base);
                            q[i] = fast_exp2(ml.x - base);
                            l[i] = l[i] * f[i] + ml.y * q[i];
                            m[i] = M;
                        }
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            const float4 y = *reinterpret_cast<const float4*>(jo + ((size_t)(at * (D / 8) + j) * 32 + lane) * 4);
                            o[j][0] = o[j][0] * f[0] + y.x * q[0];
                            o[j][1] = o[j][1] * f[0] + y.y * q[0];
                            o[j][2] = o[j][2] * f[1] + y.z * q[1];
                            o[j][3] = o[j][3] * f[1] + y.w * q[1];
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.join_empty);
                }
                return true;
            };
            const int n_ctx = (u.C + CH - 1) / CH;
            bool last = u.n < 0;
            for (; !last; ++g) {                          // the unit's own chunks
                const int st = (int)(g % C::kStages);
                if (!warp_wait(&bar.full[st], (g / C::kStages) & 1, abort, kWaitBudget)) { ok = false; break; }
                const Entry en = bar.entry[st];
                if (en.kind != 0) break;
                last = en.last != 0;
                const int c = en.c;
                if (!dead) {
                    const uint32_t kb = smem_u + st * C::kStageBytes, vb = kb + C::kKBytes;
                    float s[C::kKw / 8][4];
#pragma unroll
                    for (int j = 0; j < C::kKw / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int j = 0; j < C::kKw / 16; ++j) {
                            uint32_t kf[4];
                            ldsm4(kf, kb + (k >> 2) * (CH * 128) + sw128(k_row + 16 * j, (k & 3) * 2 + k_c));
                            mma16816(s[2 * j], qf[k], kf[0], kf[1]);
                            mma16816(s[2 * j + 1], qf[k], kf[2], kf[3]);
                        }
                    // ---- visibility: positions before the context's end, ancestor drafts
                    const bool ctx = c < n_ctx;
                    const int first = (ctx ? c : c - n_ctx) * CH + ks * C::kKw;    // this warp's first key
                    const int left = (ctx ? u.C : u.Pb) - first;                   // keys that exist
                    if (!ctx || left < C::kKw) {
                        const uint32_t in = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t bits = in;
                            if (!ctx) bits &= (first < 32 ? mw[i][0] : mw[i][1]) >> (first & 31);
                            bits >>= 2 * tc;                                       // this thread's first key
#pragma unroll
                            for (int j = 0; j < C::kKw / 8; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!((bits >> (8 * j + e)) & 1u)) s[j][2 * i + e] = -INFINITY;
                        }
                    }
                    // ---- online softmax (log2 domain), two rows a thread
                    float ms[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ms[i] = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
                        for (int j = 1; j < C::kKw / 8; ++j) ms[i] = fmaxf(ms[i], fmaxf(s[j][2 * i], s[j][2 * i + 1]));
                    }
#pragma unroll
                    for (int d = 1; d <= 2; d *= 2)
#pragma unroll
                        for (int i = 0; i < 2; ++i) ms[i] = fmaxf(ms[i], __shfl_xor_sync(0xffffffffu, ms[i], d));
                    ms[0] *= a.scale_log2;
                    ms[1] *= a.scale_log2;
                    const bool need[2] = {ms[0] > m[0] + kRescaleThreshold, ms[1] > m[1] + kRescaleThreshold};
                    if (__any_sync(0xffffffffu, need[0] || need[1])) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float f = need[i] ? fast_exp2(m[i] - ms[i]) : 1.f;   // 0 while m is -inf
                            l[i] *= f;
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                o[j][2 * i] *= f;
                                o[j][2 * i + 1] *= f;
                            }
                            if (need[i]) m[i] = ms[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float base = m[i] == -INFINITY ? 0.f : m[i];
                        float sum[2] = {0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < C::kKw / 8; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float p = fast_exp2(fmaf(s[j][2 * i + e], a.scale_log2, -base));
                                s[j][2 * i + e] = p;
                                sum[e] += p;
                            }
                        l[i] += sum[0] + sum[1];
                    }
                    // ---- O += P V, P rounded to bf16 (the product's type; l keeps 32 bits).
                    // Value rows past the end may hold anything (0 x NaN): they are cleared
                    auto pv = [&](auto ragged) {
#pragma unroll
                        for (int kk = 0; kk < C::kKw / 16; ++kk) {
                            uint32_t pf[4];
                            pf[0] = pack_bf16(s[2 * kk][0], s[2 * kk][1]);
                            pf[1] = pack_bf16(s[2 * kk][2], s[2 * kk][3]);
                            pf[2] = pack_bf16(s[2 * kk + 1][0], s[2 * kk + 1][1]);
                            pf[3] = pack_bf16(s[2 * kk + 1][2], s[2 * kk + 1][3]);
                            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                            if constexpr (decltype(ragged)::value) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int key = 16 * kk + 2 * tc + 8 * i;
                                    keep[i] = (key < left ? 0xffffu : 0u) | (key + 1 < left ? 0xffff0000u : 0u);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                uint32_t vf[4];
                                ldsm4_t(vf, vb + (j >> 2) * (CH * 128) + sw128(v_row + 16 * kk, (j & 3) * 2 + v_c));
                                if constexpr (decltype(ragged)::value) {
                                    vf[0] &= keep[0];
                                    vf[1] &= keep[1];
                                    vf[2] &= keep[0];
                                    vf[3] &= keep[1];
                                }
                                mma16816(o[2 * j], pf, vf[0], vf[1]);
                                mma16816(o[2 * j + 1], pf, vf[2], vf[3]);
                            }
                        }
                    };
                    if (left < C::kKw) pv(std::true_type{});
                    else pv(std::false_type{});
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.empty[st]);
            }
            if (!ok) break;
            if (u.n > 0 && !finish()) { ok = false; break; }
            for (; !last; ++g) {                          // its rows' partials over the prefix
                const int st = (int)(g % C::kStages);
                if (!warp_wait(&bar.full[st], (g / C::kStages) & 1, abort, kWaitBudget)) { ok = false; break; }
                const Entry en = bar.entry[st];
                last = en.last != 0;
                if (en.kind == 1 && ks == 0 && !dead) {
                    const int rows = en.r1 - en.r0;
                    if (en.half == 0) {
                        const float2* ml = reinterpret_cast<const float2*>(smem + C::kMlOff) + st * C::kMlRows + en.shift;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = rw * 16 + gr + 8 * i - en.r0;
                            const float2 x = at >= 0 && at < rows ? ml[at] : make_float2(-INFINITY, 0.f);
                            const float M = fmaxf(m[i], x.x), base = M == -INFINITY ? 0.f : M;
                            const float f = fast_exp2(m[i] - base);
                            wp[i] = fast_exp2(x.x - base);
                            l[i] = l[i] * f + x.y * wp[i];
                            m[i] = M;
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                o[j][2 * i] *= f;
                                o[j][2 * i + 1] *= f;
                            }
                        }
                    }
                    // columns [half D/2, ..): float4 [D / 8][kQRows]
                    const unsigned char* part = smem + st * C::kStageBytes;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = rw * 16 + gr + 8 * i - en.r0;
                        if (at < 0 || at >= rows) continue;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            if ((j >= D / 16) != (en.half == 1)) continue;
                            const int c4 = 2 * (j % (D / 16)) + (tc >> 1);
                            const float2 y = *reinterpret_cast<const float2*>(part + (c4 * C::kQRows + at) * 16 + (tc & 1) * 8);
                            o[j][2 * i] += y.x * wp[i];
                            o[j][2 * i + 1] += y.y * wp[i];
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.empty[st]);
            }
            if (!ok) break;
            if (ks > 0) continue;
            if (a.by_unit) {
                // ---- output rows, 16 bytes a lane (four lanes swap their pairs of columns);
                // rows behind the packed length: zeros
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = rw * 16 + gr + 8 * i;
                    const float inv = row < live && l[i] != 0.f ? 1.f / l[i] : 0.f;
                    uint4* dst = reinterpret_cast<uint4*>(
                        a.o + ((size_t)(u.row0 + row / a.G) * a.Hq + u.h * a.G + row % a.G) * D);
#pragma unroll
                    for (int j0 = 0; j0 < D / 8; j0 += 4) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = row < live ? pack_bf16(o[j0 + k][2 * i] * inv, o[j0 + k][2 * i + 1] * inv) : 0u;
                        swap4(v, tc);
                        if (row < u.rows >> 16) dst[j0 + tc] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
                continue;
            }
            // ---- fp32 partials, float4 [D / 4][rows]: eight rows' column pairs make
            // whole lines
            const bool whole = u.slot < 0;
            const size_t stride = whole ? a.p.suffix.rows_cap : (size_t)a.p.slot_rows;
            const size_t block = whole ? u.h : u.slot;
            float* dst = reinterpret_cast<float*>((whole ? a.p.suffix.rows : a.p.suf_part) + block * (D / 4) * stride);
            float2* dml = (whole ? a.p.suffix.rows_ml : a.p.suf_part_ml) + block * stride;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = rw * 16 + gr + 8 * i;
                if (row >= live) continue;
                const size_t at = whole ? (size_t)u.row0 * a.G + row : (size_t)row;
#pragma unroll
                for (int j = 0; j < D / 8; ++j)           // columns 8 j + 2 tc, + 1
                    *reinterpret_cast<float2*>(dst + (((size_t)(2 * j + (tc >> 1))) * stride + at) * 4 + (tc & 1) * 2) =
                        make_float2(o[j][2 * i], o[j][2 * i + 1]);
                if (tc == 0) dml[at] = make_float2(m[i], l[i]);
            }
        }
        if (!ok) fail();
        // this grid's end has to mean the prefix's too (the merge waits for this grid).
        // One whole warp waits: in the producer's warp the idle lanes would, and hold
        // up the lane that loads until the prefix has ended
        if (warp == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    }
}

// [rows, heads, D] bf16 -> boxes of `pos` rows x `heads_box` heads x 64 columns
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int D, int heads_box, int pos)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)pos};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// partials: float4 [blocks][D / 4][rows] -> boxes of `box` rows x D / 8 column groups
bool make_partial_map(CUtensorMap* map, const void* base, size_t rows, size_t groups, int box, int D)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)rows * 4, (cuuint64_t)groups};
    cuuint64_t strides[1] = {(cuuint64_t)rows * 16};
    cuuint32_t boxes[2] = {(cuuint32_t)box * 4, (cuuint32_t)D / 8};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, boxes, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NW, int KS>
cudaError_t launch(int grid, cudaStream_t stream, SuffixArgs& a, CUtensorMap* m)
{
    using C = SCfg<D, NW, KS>;
    cudaError_t e = cudaFuncSetAttribute(suffix_kernel<D, NW, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmemBytes);
    if (e != cudaSuccess) return e;
    void* args[] = {&a, &m[0], &m[1], &m[2], &m[3], &m[4], &m[5], &m[6]};
    return launch_dependent(reinterpret_cast<const void*>(suffix_kernel<D, NW, KS>), dim3(grid), dim3(C::kThreads),
                            C::kSmemBytes, stream, args);
}

template <int D>
cudaError_t launch_rows(int grid, cudaStream_t stream, SuffixArgs& a, CUtensorMap* m)
{
    switch (rd_suffix_row_warps(a.nodes * a.G)) {
    case 1: return launch<D, 1, 4>(grid, stream, a, m);
    case 2: return launch<D, 2, 2>(grid, stream, a, m);
    case 3: return launch<D, 3, 1>(grid, stream, a, m);
    default: return launch<D, 4, 1>(grid, stream, a, m);
    }
}

}  // namespace

// Whole units off a counter when they are many enough to level out: 64 and 128 units
// (one token of 8 requests, up to 20 nodes of 4) make the whole call 33 and 42 us that way,
// 23 and 28 in ranges; 2,560 units 262 us against 277 with partials and a merge.
bool rd_suffix_by_unit(long long units, int grid) { return units >= 4LL * grid; }

int rd_suffix_grid(int rows) { return rd_device_sm_count() * rd_suffix_ctas(rd_suffix_row_warps(rows)); }

cudaError_t rd_launch_shared_suffix(const rdshared::Plan& p, int B, int P_max, int Hq, int Hkv, int D,
                                    float scale_log2, const void* q, const void* k_new, const void* v_new,
                                    const void* k_pool, const void* v_pool, const rd_paged_kv& paged,
                                    const uint32_t* mask, int mask_words, bool by_unit, void* o, int32_t* dev_status,
                                    cudaStream_t stream)
{
    SuffixArgs a = {};
    a.B = B;
    a.P_max = P_max;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.page_size = paged.page_size;
    a.max_pages = paged.max_pages;
    a.num_pages = paged.num_pages;
    a.mask_words = mask_words;
    a.scale_log2 = scale_log2;
    a.block_table = paged.block_table;
    a.ctx_lens = paged.ctx_lens;
    a.mask = mask;
    a.p = p;
    a.o = static_cast<uint16_t*>(o);
    a.by_unit = by_unit;
    a.status = dev_status;
    a.stall_budget = rd_attention_stall_budget();
    a.nodes = rd_suffix_nodes(P_max, a.G);
    a.blocks = (P_max + a.nodes - 1) / a.nodes;
    const int rows = a.nodes * a.G, ch = rd_suffix_chunk(rd_suffix_row_warps(rows));
    const int64_t pool_rows = (int64_t)paged.num_pages * paged.page_size, new_rows = (int64_t)B * P_max;
    CUtensorMap m[7];
    const int box = rd_suffix_row_warps(rows) * 16;
    if (!make_map(&m[0], k_pool, pool_rows, Hkv, D, 1, ch) || !make_map(&m[1], v_pool, pool_rows, Hkv, D, 1, ch) ||
        !make_map(&m[2], k_new, new_rows, Hkv, D, 1, ch) || !make_map(&m[3], v_new, new_rows, Hkv, D, 1, ch) ||
        !make_map(&m[4], q, new_rows, Hq, D, a.G, a.nodes))
        return cudaErrorInvalidValue;
    if (by_unit) {
        if (!make_partial_map(&m[5], p.rows, p.rows_cap, (size_t)Hkv * (D / 4), box, D) ||
            !make_partial_map(&m[6], p.part, kUnitRows, (size_t)2 * p.grid * (D / 4), box, D))
            return cudaErrorInvalidValue;
    } else {
        m[5] = m[6] = m[0];                               // not used
    }
    const int grid = rd_suffix_grid(rows);
    return D == 128 ? launch_rows<128>(grid, stream, a, m) : launch_rows<64>(grid, stream, a, m);
}
