// rd_tree_attention_quant: tree attention over a paged cache held in 4 or in 8 bits
// (quant_format.cuh), single-token decoding among it.
//
//   o[r] = sum_j softmax_j(scale q[r] . k[j]) v[j]
//
// over the context (all visible) and the packed drafts (ancestors and the node itself), in one
// pass with a running maximum and sum.  What it must read is half to a quarter of the 16-bit
// cache, so widening the codes, not the stream, is the nearest bound: per position and kv
// head 2 D codes become 16-bit floats.  Each code is widened once per unit's rows, in the registers
// that feed the matrix instructions, with no way through shared memory:
//
//   S^T[16 positions x 8 rows] += K[16 x 16] Q^T[16 x 8]      A = K, straight from the codes
//   O^T[16 columns x 8 rows]   += V^T[16 x 16] P^T[16 x 8]    A = V^T, straight from the codes
//
// The order in which a contraction runs is free, so a thread takes 16 consecutive elements
// of a row of K (one block, one scale) as its share of four steps, and V's columns are dealt
// so that a thread owns 16 consecutive ones: its loads are whole blocks and its outputs whole
// 16-byte words.  Rows are the products' short side: 8 at a time, so that five rows cost a
// quarter of what 32 do.
//
// 64 contexts of 8,192 with 23 nodes of 48 and 40 heads take 1,141 us (2.6 TB/s of codes): the matrix
// unit, one of these products every two cycles, is busy for 490 of them, and the 8 warps that the registers leave room
// for do not hide each other's chains (code to float, product, exponential, product) any better.
// A call of one short piece a CTA is its start and end: 8 tokens of 2,000 positions take 20.6 us, 16 of them for
// the division of the work, the walk to the piece, the queries, a slow first chunk, the join and the merge.
#include "quant_attention.cuh"

namespace {

using namespace rdquant;

// Warps that compute: the sums of 32 rows take 128 registers of a thread with D = 128, which leaves room for
// 8; with D = 64 12 fit, and hide more of each other's latency.
constexpr int warps_of(int D) { return D == 128 ? 8 : 12; }
constexpr int kLoaders = 4;                // warps that load
constexpr int threads_of(int D) { return 32 * (warps_of(D) + kLoaders); }
// registers of a thread: the launch's (all of an SM's), dealt anew
constexpr int launch_regs(int D) { return D == 128 ? 168 : 128; }
constexpr int compute_regs(int D) { return D == 128 ? 232 : 152; }
constexpr int load_regs(int D) { return D == 128 ? 40 : 56; }
constexpr bool regs_fit(int D)
{
    return 32 * (warps_of(D) * compute_regs(D) + kLoaders * load_regs(D)) <= threads_of(D) * launch_regs(D);
}
static_assert(regs_fit(64) && regs_fit(128), "registers");
// rows of a unit at most (with D = 64, 32 rows spill from 152 registers: two contexts of 50,000 74 us, not 51)
constexpr int kMostRows = 32;
constexpr int rows_of(int D) { return D == 128 ? kMostRows : 24; }
// tiles of 16 positions of a warp's share of a chunk (the ring holds few chunks of 8-bit rows of 128)
constexpr int tiles_of(int D, int bits) { return D == 128 && bits == 8 ? 1 : 2; }
constexpr int kDraftTile = 16;             // packed drafts of a chunk
constexpr int kMostStages = 8;
// positions of a TMA box: chunks of 96 positions are no whole number of 64
constexpr int box_of(int D, int bits) { return tiles_of(D, bits) * warps_of(D) % 16 == 0 ? 64 : 32; }

struct Shared {                            // static part
    uint64_t full[kMostStages], empty[kMostStages], never;
    int abort, never_abort;
    DivisionShared division;
};

// a place in the ring
struct Turn {
    int stage;
    uint32_t parity;           // of the stage's phase
    __device__ __forceinline__ void next(int stages)
    {
        if (++stage == stages) {
            stage = 0;
            parity ^= 1u;
        }
    }
};

// ------------------------------------------------------------------ small pieces of PTX
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int D>
__device__ __forceinline__ void compute_sync() { rdtc::named_sync(1, 32 * warps_of(D)); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// ------------------------------------------------------------------ loading
// The positions of a warp's tile are dealt to the products' indices so that both the four
// rows of K and the four rows of V that a half-warp reads lie in different banks.
__device__ __forceinline__ int position_of(int t, int e) { return 4 * e + ((t + 2 * e) & 3); }    // e: 0, 1

template <int BYTES>
__device__ __forceinline__ void load_rows(const Args& a, uint32_t k_to, uint32_t v_to, const size_t (&base)[6], int rows,
                                          int tid)
{
    const size_t row = (size_t)a.Hkv * a.seg / a.heads;
    const int copies = rows * a.per_row;
    for (int i = tid; i < copies; i += 32 * kLoaders) {
        const int pos = (int)__umulhi((uint32_t)i, a.per_row_magic), part = i - pos * a.per_row;
        const int blk = pos >> 6;
        size_t at0 = base[0];
#pragma unroll
        for (int k = 1; k < 6; ++k) at0 = blk == k ? base[k] : at0;
        const size_t at = at0 + (size_t)(pos & 63) * row + (size_t)part * BYTES;
        const uint32_t to = (uint32_t)(pos * a.pitch + part * BYTES);
        copy_async<BYTES>(k_to + to, a.k_pool + at);
        copy_async<BYTES>(v_to + to, a.v_pool + at);
    }
}

// One warp fetches everything by TMA: a box of 64 or 32 positions x the unit's heads (for 8 bits one
// for each 128 bytes of them, swizzled) per pool, the drafts' rows as bulk copies.  Lane k has the k-th
// box of a chunk, and reads the next chunk's entry of the table while this one's copies go out: the
// warp's time per chunk is what bounds small rows (without this, 1,500 cycles for 32 positions).
template <int D, int BITS>
__device__ __forceinline__ void load_tiled(const Args& a, Shared& sh, unsigned char* ring, const Division& d)
{
    const int lane = threadIdx.x & 31, chunk = a.chunk, box = box_of(D, BITS);
    const bool mine = lane * box < chunk;
    Walk walk = Walk::over(a, d);
    Piece p;
    Turn at = {0, 1};                      // (an empty stage's first phase counts as done)
    bool alive = true;
    uint32_t filled = 0;
    while (alive && walk.next(a, p)) {
        const int32_t* table = a.table + (size_t)p.b * a.max_pages;
        // (Positions of chunks of drafts and of idle lanes lie up to 5,200 behind the context's end, which may be
        // 2^31 - 257: unsigned, and from there on how many are left.)
        const uint32_t pos = (uint32_t)p.j0 * chunk + lane * box;
        int left = (int)((uint32_t)p.C - pos), in_page = (int)(pos % (uint32_t)a.page_size);
        table += pos / (uint32_t)a.page_size;
        int page = mine && left > 0 ? __ldg(table) : 0;
        const int x = p.hg * (a.seg / 4);
        for (int j = p.j0; j < p.j1; ++j) {
            unsigned char* k_to = ring + (size_t)at.stage * 2 * a.half;
            unsigned char* v_to = k_to + a.half;
            uint64_t* bar = &sh.full[at.stage];
            uint64_t* empty = &sh.empty[at.stage];
            if (j < p.n_ctx) {
                const bool live = mine && left > 0;
                const int boxes = __popc(__ballot_sync(0xffffffffu, live));
                if (live && (page < 0 || page >= a.num_pages)) {
                    rd_flag(a.status, RD_DEV_BAD_INDEX);
                    page = 0;
                }
                const int row = page * a.page_size + in_page;            // (31 bits: see launch)
                left -= chunk;
                for (in_page += chunk; in_page >= a.page_size; in_page -= a.page_size) ++table;
                page = mine && left > 0 ? __ldg(table) : 0;
                alive = rdattn::warp_wait(empty, at.parity, &sh.abort, kWaitBudget);
                if (!alive) break;         // nobody waits for copies any more
                if (lane == 0) rdtc::mbar_arrive_expect_tx(bar, (uint32_t)(2 * boxes * box * a.seg));
                __syncwarp();
                if (live) {
                    if constexpr (BITS == 4) {
                        const size_t to = (size_t)lane * box * a.seg;
                        rdtc::tma_load_2d(k_to + to, &a.k_map, bar, x, row);
                        rdtc::tma_load_2d(v_to + to, &a.v_map, bar, x, row);
                    } else {
                        for (int i = 0; i < a.seg / 128; ++i) {
                            const size_t to = ((size_t)i * chunk + lane * box) * 128;
                            rdtc::tma_load_2d(k_to + to, &a.k_map, bar, x + 32 * i, row);
                            rdtc::tma_load_2d(v_to + to, &a.v_map, bar, x + 32 * i, row);
                        }
                    }
                }
            } else {
                alive = rdattn::warp_wait(empty, at.parity, &sh.abort, kWaitBudget);
                if (!alive) break;
                const int node0 = (j - p.n_ctx) * kDraftTile, nodes = min(kDraftTile, p.len - node0), bytes = a.heads * D * 2;
                if (lane == 0) rdtc::mbar_arrive_expect_tx(bar, (uint32_t)(2 * nodes * bytes));
                __syncwarp();
                if (lane < nodes) {
                    const size_t from = (((size_t)p.b * a.P + node0 + lane) * a.Hkv + (size_t)p.hg * a.heads) * D;
                    rdtc::bulk_load(k_to + lane * a.draft_pitch, a.k_new + from, (uint32_t)bytes, bar);
                    rdtc::bulk_load(v_to + lane * a.draft_pitch, a.v_new + from, (uint32_t)bytes, bar);
                }
            }
            __syncwarp();
            at.next(a.stages);
            ++filled;
        }
    }
    // no copy may be under way when the CTA ends: the last stages' have all landed
    const uint32_t stages = (uint32_t)a.stages;
    for (uint32_t i = filled > stages ? filled - stages : 0; i < filled; ++i)
        rdattn::warp_wait(&sh.full[i % stages], (i / stages) & 1u, &sh.never_abort, kWaitBudget);
}

// The same by 128 threads with copies of 16, 8 or 4 bytes, for rows that TMA's rules leave out (an
// odd number of kv heads).
template <int D, int BITS>
__device__ __forceinline__ void load_rowwise(const Args& a, Shared& sh, unsigned char* ring, const Division& d)
{
    const int chunk = a.chunk;
    const int tid = threadIdx.x - 32 * warps_of(D);
    const int64_t row = (int64_t)a.Hkv * a.seg / a.heads;
    Walk walk = Walk::over(a, d);
    Piece p;
    uint32_t it = 0;
    bool alive = true;
    while (walk.next(a, p)) {
        for (int j = p.j0; j < p.j1; ++j, ++it) {
            const int stage = (int)(it % (uint32_t)a.stages);
            // where the positions lie, before the wait
            size_t base[6] = {0, 0, 0, 0, 0, 0};
            int rows = 0;
            if (j < p.n_ctx) {
                const int pos0 = j * chunk;
                rows = min(chunk, p.C - pos0);
#pragma unroll
                for (int k = 0; k < 6; ++k)
                    if (64 * k < rows) base[k] = (size_t)(row_at(a, p.b, pos0 + 64 * k, tid == 0) * row + (int64_t)p.hg * a.seg);
            }
            if (alive && it >= (uint32_t)a.stages)
                alive = rdattn::warp_wait(&sh.empty[stage], ((it / (uint32_t)a.stages) & 1u) ^ 1u, &sh.abort, kWaitBudget);
            const uint32_t k_to = smem_addr(ring + (size_t)stage * 2 * a.half), v_to = k_to + (uint32_t)a.half;
            if (j < p.n_ctx) {
                if (a.gran == 16) load_rows<16>(a, k_to, v_to, base, rows, tid);
                else if (a.gran == 8) load_rows<8>(a, k_to, v_to, base, rows, tid);
                else load_rows<4>(a, k_to, v_to, base, rows, tid);
            } else {
                const int node0 = (j - p.n_ctx) * kDraftTile;
                const int nodes = min(kDraftTile, p.len - node0);
                const int copies = a.heads * D * 2 / 16;
                for (int i = tid; i < nodes * copies; i += 32 * kLoaders) {
                    const int node = i / copies, part = i % copies;
                    const size_t at = (((size_t)p.b * a.P + node0 + node) * a.Hkv + (size_t)p.hg * a.heads) * D + (size_t)part * 8;
                    const uint32_t to = (uint32_t)(node * a.draft_pitch + part * 16);
                    copy_async<16>(k_to + to, a.k_new + at);
                    copy_async<16>(v_to + to, a.v_new + at);
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sh.full[stage])) : "memory");
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// rows behind the last node, and those of skipped requests
template <int D>
__device__ __forceinline__ void clear_rows(const Args& a)
{
    const int tid = threadIdx.x - 32 * warps_of(D);
    const int vecs = a.Hq * D / 8;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int from = shape_of(a, b).len;
        uint4* o = reinterpret_cast<uint4*>(a.o) + (size_t)b * a.P * vecs;
        for (size_t v = (size_t)from * vecs + tid; v < (size_t)a.P * vecs; v += 32 * kLoaders) o[v] = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ computing
// What a warp needs to know of its place.
struct Place {
    int warp, lane, g, t;      // lane = 4 g + t
    int head, split, splits;   // kv head within the group, share of each chunk's positions
};

template <int D, int BITS, int NT>
struct Sums {                              // of 8 NT rows; this thread's columns D / 8 * g ..., rows 8 i + 2 t, + 1
    float o[D / 16][NT][4];
    uint32_t none;                         // bit k: row k has no reference yet
    bool fresh;                            // some row of the warp has none
    // A thread's factors, references and sums of weights lie in shared memory: its registers are taken.
    uint32_t fr, l;
    __device__ __forceinline__ float reference(int k) const { return -__uint_as_float(lds32(fr + (uint32_t)(64 * (k / 2) + 8 * (k & 1) + 4))); }
    __device__ __forceinline__ void set_reference(int k, float r) const
    {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(fr + (uint32_t)(64 * (k / 2) + 8 * (k & 1) + 4)), "f"(-r) : "memory");
    }
    __device__ __forceinline__ void sums(float (&v)[2 * NT]) const
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint2 u = lds64(l + (uint32_t)(256 * i));
            v[2 * i] = __uint_as_float(u.x), v[2 * i + 1] = __uint_as_float(u.y);
        }
    }
    __device__ __forceinline__ void set_sums(const float (&v)[2 * NT]) const
    {
#pragma unroll
        for (int i = 0; i < NT; ++i)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(l + (uint32_t)(256 * i)), "f"(v[2 * i]), "f"(v[2 * i + 1]) : "memory");
    }
};

// maximum (or sum) over the lanes that share a row
template <int NT, bool SUM>
__device__ __forceinline__ void over_lanes(float (&v)[2 * NT])
{
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, v[k], o);
            v[k] = SUM ? v[k] + x : fmaxf(v[k], x);
        }
}

// new references, kBelow under the rows' maxima: `top` is this thread's
template <int D, int BITS, int NT>
__device__ __forceinline__ void raise(Sums<D, BITS, NT>& s, float (&top)[2 * NT])
{
    // (No lane may leave the common way here: rows without a reference differ from lane to lane.)
    uint32_t none = 0;
    float l[2 * NT];
    over_lanes<NT, false>(top);
    s.sums(l);
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) {
        const float v = top[k] - kBelow, was = s.reference(k);
        const bool had = !(s.none >> k & 1u), still = v == -INFINITY && !had;
        top[k] = had ? fmaxf(was, v) : still ? 0.f : v;
        const float f = had ? fast_exp2(was - top[k]) : 0.f;         // (nothing summed yet)
        none |= still ? 1u << k : 0u;
        l[k] *= f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            s.o[j][k / 2][k & 1] *= f;
            s.o[j][k / 2][2 + (k & 1)] *= f;
        }
    }
    s.set_sums(l);
    __syncwarp();                                      // all have read the old references
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) s.set_reference(k, top[k]);     // (lanes that share a row agree)
    __syncwarp();
    s.none = none;
    s.fresh = __any_sync(0xffffffffu, none != 0);
}

// Byte `at` of the row of position `pos` (of this warp's tile) within a stage.
template <int BITS>
struct Rows {
    uint32_t base;             // of the tile's first position
    int pitch;
    uint32_t first;            // byte of the head's row within 128 bytes (8 bits, swizzled)
    bool swizzled;
    __device__ __forceinline__ uint32_t operator()(int pos, int at) const
    {
        if constexpr (BITS == 4) return base + (uint32_t)(pos * pitch + at);
        const uint32_t x = first + (uint32_t)at;
        return base + (uint32_t)(pos * pitch) + (swizzled ? x ^ (uint32_t)((pos & 7) << 4) : x);
    }
};

// MT tiles of 16 positions of the context; `valid` of them count
template <int D, int BITS, int NT, int MT>
__device__ __forceinline__ void context_tiles(const Args& a, const Place& w, Sums<D, BITS, NT>& s, const Rows<BITS>& k_row,
                                              const Rows<BITS>& v_row, uint32_t q_at, int valid)
{
    using namespace rdquant;
    constexpr int KB = D / 64;             // blocks of a row of K that a thread widens
    float x[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[m][i][c] = 0.f;
    const int pos = position_of(w.g >> 1, w.g & 1);
    // ---- S^T
    uint32_t sc[MT][2][KB];
    if constexpr (BITS == 4) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t at = k_row(16 * m + pos + 8 * e, D / 2);
                if constexpr (D == 128) {
                    const uint2 b = lds64(at);
                    e4m3x4(__byte_perm(b.x, b.y, (uint32_t)w.t * 0x1111u + 0x4400u), sc[m][e][0], sc[m][e][KB - 1]);
                } else {
                    uint32_t drop;
                    e4m3x4(__byte_perm(lds32(at), 0u, (uint32_t)w.t * 0x1111u), sc[m][e][0], drop);
                }
            }
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        uint32_t c[MT][2][BITS == 4 ? 2 : 4];          // the thread's 16 codes of each of its positions
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t at = k_row(16 * m + pos + 8 * e, (BITS == 4 ? 8 : 16) * (w.t + 4 * kb));
                if constexpr (BITS == 8) {
                    const uint4 u = lds128(at);
                    c[m][e][0] = u.x, c[m][e][1] = u.y, c[m][e][BITS == 8 ? 2 : 0] = u.z, c[m][e][BITS == 8 ? 3 : 0] = u.w;
                } else if constexpr (D == 128) {
                    const uint2 u = lds64(at);
                    c[m][e][0] = u.x, c[m][e][1] = u.y;
                } else {
                    c[m][e][0] = lds32(at), c[m][e][1] = lds32(at + 4);
                }
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {      // two steps of 16 at a time
            uint32_t f[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (BITS == 4) {
                        uint32_t v[4];
                        e2m1x8(c[m][e][h], v);
                        f[m][0][e] = mul_f16x2(v[0], sc[m][e][kb]);
                        f[m][0][2 + e] = mul_f16x2(v[1], sc[m][e][kb]);
                        f[m][1][e] = mul_f16x2(v[2], sc[m][e][kb]);
                        f[m][1][2 + e] = mul_f16x2(v[3], sc[m][e][kb]);
                    } else {
                        e4m3x4(c[m][e][2 * h], f[m][0][e], f[m][0][2 + e]);
                        e4m3x4(c[m][e][2 * h + 1], f[m][1][e], f[m][1][2 + e]);
                    }
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint2 qb = lds64(q_at + (uint32_t)(i * 8 * (2 * D + 16) + 128 * kb + 16 * h));
#pragma unroll
                for (int m = 0; m < MT; ++m) mma_f16(x[m][i], f[m][0], qb.x, qb.y);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint2 qb = lds64(q_at + (uint32_t)(i * 8 * (2 * D + 16) + 128 * kb + 16 * h + 8));
#pragma unroll
                for (int m = 0; m < MT; ++m) mma_f16(x[m][i], f[m][1], qb.x, qb.y);
            }
        }
    }
    // ---- softmax of the rows over these positions
    if (valid < 16 * MT) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (16 * m + pos >= valid) x[m][i][0] = x[m][i][1] = -INFINITY;
                if (16 * m + pos + 8 >= valid) x[m][i][2] = x[m][i][3] = -INFINITY;
            }
    }
    // exponents over the references; one above kBelow + kLag, or a row without a reference, needs new ones
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint4 v = lds128(s.fr + (uint32_t)(64 * i));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[m][i][c] = fmaf(x[m][i][c], __uint_as_float(c & 1 ? v.z : v.x), __uint_as_float(c & 1 ? v.w : v.y));
                most = fmaxf(most, x[m][i][c]);
            }
    }
    if (__any_sync(0xffffffffu, most > kBelow + kLag) || s.fresh) {
        float top[2 * NT];
#pragma unroll
        for (int k = 0; k < 2 * NT; ++k) {
            const float was = s.reference(k);
            top[k] = -INFINITY;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                x[m][k / 2][k & 1] += was;
                x[m][k / 2][2 + (k & 1)] += was;
                top[k] = fmaxf(top[k], fmaxf(x[m][k / 2][k & 1], x[m][k / 2][2 + (k & 1)]));
            }
        }
        raise<D, BITS, NT>(s, top);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[m][i][c] -= top[2 * i + (c & 1)];
    }
    float l[2 * NT];
    s.sums(l);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) p[c] = fast_exp2(x[m][i][c]);
            l[2 * i] += p[0] + p[2];
            l[2 * i + 1] += p[1] + p[3];
            pb[i][0] = transpose8x8(pack_f16(p[0], p[1]));       // 2^-11 of each weight
            pb[i][1] = transpose8x8(pack_f16(p[2], p[3]));
        }
        if (m == MT - 1) s.set_sums(l);
        // ---- O^T
        const int first = 16 * m, v[4] = {first + position_of(w.t, 0), first + position_of(w.t, 1),
                                          first + position_of(w.t, 0) + 8, first + position_of(w.t, 1) + 8};
        if constexpr (BITS == 4) {
            constexpr int NW = D / 64;     // words of the thread's columns
            uint32_t u[4][NW], b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (D == 128) {
                    const uint2 y = lds64(v_row(v[e], 8 * w.g));
                    u[e][0] = y.x, u[e][NW - 1] = y.y;
                    b[e] = lds8(v_row(v[e], D / 2 + w.g));
                } else {
                    u[e][0] = lds32(v_row(v[e], 4 * w.g));
                    b[e] = lds8(v_row(v[e], D / 2 + (w.g >> 1)));
                }
                // what lies behind the end may be anything: its scale is 0
                if (valid < 16 * MT && v[e] >= valid) b[e] = 0;
            }
            uint32_t s01, s23;
            e4m3x4(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, s01, s23);
#pragma unroll
            for (int q = 0; q < NW; ++q) {
                // the codes of one column at two positions, side by side
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                uint32_t e0[4], o0[4], e1[4], o1[4];
                e2m1x8((u[0][q] & kLow) | ((u[1][q] << 4) & ~kLow), e0);
                e2m1x8(((u[0][q] >> 4) & kLow) | (u[1][q] & ~kLow), o0);
                e2m1x8((u[2][q] & kLow) | ((u[3][q] << 4) & ~kLow), e1);
                e2m1x8(((u[2][q] >> 4) & kLow) | (u[3][q] & ~kLow), o1);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t f[4] = {mul_f16x2(e0[c], s01), mul_f16x2(o0[c], s01), mul_f16x2(e1[c], s23),
                                           mul_f16x2(o1[c], s23)};
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_f16(s.o[4 * q + c][i], f, pb[i][0], pb[i][1]);
                }
            }
        } else {
            constexpr int NW = D / 32;
            uint32_t u[4][NW];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t at = v_row(v[e], D / 8 * w.g);
                if constexpr (D == 128) {
                    const uint4 y = lds128(at);
                    u[e][0] = y.x, u[e][1] = y.y, u[e][NW - 2] = y.z, u[e][NW - 1] = y.w;
                } else {
                    const uint2 y = lds64(at);
                    u[e][0] = y.x, u[e][1] = y.y;
                }
                if (valid < 16 * MT && v[e] >= valid) {
#pragma unroll
                    for (int q = 0; q < NW; ++q) u[e][q] = 0;
                }
            }
#pragma unroll
            for (int q = 0; q < NW; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h == 0 ? 0x5140u : 0x7362u;
                    uint32_t f[4];
                    e4m3x4(__byte_perm(u[0][q], u[1][q], sel), f[0], f[1]);
                    e4m3x4(__byte_perm(u[2][q], u[3][q], sel), f[2], f[3]);
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_f16(s.o[2 * q + h][i], f, pb[i][0], pb[i][1]);
                }
        }
    }
}

__device__ __forceinline__ uint32_t bf16_of_f16(uint32_t x)
{
    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&x));
    return pack_bf16(v.x, v.y);
}

// one tile of 16 packed drafts: bf16 as they are; P is rounded to bf16 too (both factors of
// a product have one type), 2^-8 of each weight
template <int D, int BITS, int NT>
__device__ __forceinline__ void draft_tile(const Args& a, const Place& w, const Piece& pc, Sums<D, BITS, NT>& s, uint32_t k_at,
                                           uint32_t v_at, uint32_t q_at, uint32_t f_at, int node0, int nodes)
{
    constexpr int KB = D / 64;
    float x[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[i][c] = 0.f;
    const int pos = position_of(w.g >> 1, w.g & 1);
    // which of the rows' mask bits are these nodes'
    uint32_t seen[2 * NT];
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) {
        const int r = 8 * (k / 2) + 2 * w.t + (k & 1);
        seen[k] = 0;
        if (r < pc.rows)
            seen[k] = a.mask[((size_t)pc.b * a.P + (pc.r0 + r) / a.G) * a.mask_words + node0 / 32] >> (node0 % 32);
        if (nodes < 16) seen[k] &= (1u << nodes) - 1u;
    }
    const uint32_t row0 = k_at + (uint32_t)(pos * a.draft_pitch), row1 = row0 + (uint32_t)(8 * a.draft_pitch);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t off = (uint32_t)(32 * (w.t + 4 * kb) + 16 * h);
            const uint4 y0 = lds128(row0 + off), y1 = lds128(row1 + off);
            const uint32_t f0[4] = {y0.x, y1.x, y0.y, y1.y}, f1[4] = {y0.z, y1.z, y0.w, y1.w};
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 qb = lds128(q_at + (uint32_t)(i * 8 * (2 * D + 16) + 128 * kb + 16 * h));
                mma_bf16(x[i], f0, bf16_of_f16(qb.x), bf16_of_f16(qb.y));
                mma_bf16(x[i], f1, bf16_of_f16(qb.z), bf16_of_f16(qb.w));
            }
        }
    float top[2 * NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint2 u = lds64(f_at + (uint32_t)(32 * i));
        const float f[2] = {__uint_as_float(u.x), __uint_as_float(u.y)};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            x[i][c] = (seen[2 * i + (c & 1)] >> (pos + 4 * (c & 2)) & 1u) ? x[i][c] * f[c & 1] : -INFINITY;
        top[2 * i] = fmaxf(x[i][0], x[i][2]);
        top[2 * i + 1] = fmaxf(x[i][1], x[i][3]);
    }
    raise<D, BITS, NT>(s, top);
    uint32_t pb[NT][2];
    float l[2 * NT];
    s.sums(l);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const float p0 = fast_exp2(x[i][0] - top[2 * i]), p1 = fast_exp2(x[i][1] - top[2 * i + 1]);
        const float p2 = fast_exp2(x[i][2] - top[2 * i]), p3 = fast_exp2(x[i][3] - top[2 * i + 1]);
        l[2 * i] += p0 + p2;
        l[2 * i + 1] += p1 + p3;
        pb[i][0] = transpose8x8(pack_bf16(p0 * a.v_down, p1 * a.v_down));
        pb[i][1] = transpose8x8(pack_bf16(p2 * a.v_down, p3 * a.v_down));
    }
    s.set_sums(l);
    const int v[4] = {position_of(w.t, 0), position_of(w.t, 1), position_of(w.t, 0) + 8, position_of(w.t, 1) + 8};
#pragma unroll
    for (int part = 0; part < D / 64; ++part) {           // eight columns at a time
        uint4 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = v[e] < nodes ? lds128(v_at + (uint32_t)(v[e] * a.draft_pitch + D / 4 * w.g + 16 * part)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = q == 0 ? y[e].x : q == 1 ? y[e].y : q == 2 ? y[e].z : y[e].w;
            const uint32_t f[4] = {__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[0], z[1], 0x7632),
                                   __byte_perm(z[2], z[3], 0x5410), __byte_perm(z[2], z[3], 0x7632)};
#pragma unroll
            for (int i = 0; i < NT; ++i) mma_bf16(s.o[4 * part + q][i], f, pb[i][0], pb[i][1]);
        }
    }
}

struct Buffers {
    unsigned char* ring;
    __half* q;                 // [heads][rows][D + 8]
    float* f;                  // [heads][rows] score of a cached key = product x f (log2 units, the cache's scale in it)
    float* f_new;              // [heads][rows] the same of a draft
    float2* fr;                // [warps][rows] f, and minus the row's reference
    float2* l;                 // [warps][rows / 8][32] each thread's sums of weights
    float4* join;              // [warps / 2][2][D / 16][32]
    float2* join_ml;           // [warps / 2][8][32]
};

// m 2^e with m in [1, 2], e taken to the nearest exponent that a number has.  Never 0, which times the -inf of what lies
// behind the context's end is no number: no score moves by as much as 2^-90.
__device__ __forceinline__ float factor(float m, int e) { return m * __uint_as_float((uint32_t)min(max(e + 127, 1), 253) << 23); }

// The queries of a unit as 16-bit floats.  A power of two per row brings its largest element to
// [2^14, 2^15): elements down to 2^-28 of it stay exact, and no finite query leaves the range.
template <int D>
__device__ __forceinline__ void stage_queries(const Args& a, const Place& w, const Piece& p, const Buffers& buf, int tiles)
{
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    const int sub = w.lane % kLanes;
    const int h = p.hg * a.heads + w.head;
    for (int r = w.split * kAtOnce + w.lane / kLanes; r < 8 * tiles; r += w.splits * kAtOnce) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
            const int row = p.r0 + r;
            v = *(reinterpret_cast<const uint4*>(
                      a.q + (((size_t)p.b * a.P + row / a.G) * a.Hq + (size_t)h * a.G + row % a.G) * D) + sub);
        }
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float x[8], top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
            top = fmaxf(top, fabsf(x[e]));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = (int)(__float_as_uint(top) >> 23);
        const int k = top == 0.f || e == 255 ? 127 : min(240, 268 - e);
        const float up = __uint_as_float((uint32_t)k << 23);
        uint4 out;
        out.x = pack_f16(x[0] * up, x[1] * up);
        out.y = pack_f16(x[2] * up, x[3] * up);
        out.z = pack_f16(x[4] * up, x[5] * up);
        out.w = pack_f16(x[6] * up, x[7] * up);
        *reinterpret_cast<uint4*>(buf.q + ((size_t)w.head * rows_of(D) + r) * (D + 8) + 8 * sub) = out;
        if (sub == 0) {
            buf.f[w.head * rows_of(D) + r] = factor(a.ctx_m, a.ctx_e + 127 - k);
            buf.f_new[w.head * rows_of(D) + r] = factor(a.new_m, a.new_e + 127 - k);
        }
    }
}

template <int D, int BITS, int NT>
__device__ __forceinline__ void piece(const Args& a, Shared& sh, const Buffers& buf, const Place& w, const Piece& p,
                                      Turn& at, bool& alive)
{
    constexpr int TILES = tiles_of(D, BITS);
    const int chunk = a.chunk;
    Sums<D, BITS, NT> s;
    s.none = (1u << 2 * NT) - 1u;
    s.fr = smem_addr(buf.fr + w.warp * rows_of(D) + 2 * w.t);
    s.l = smem_addr(buf.l + w.warp * (rows_of(D) / 8) * 32 + w.lane);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s.o[j][i][c] = 0.f;
    s.fresh = true;
    compute_sync<D>();                        // nobody reads the last piece's queries any more
    stage_queries<D>(a, w, p, buf, NT);
    compute_sync<D>();
    const uint32_t q_at = smem_addr(buf.q) + (uint32_t)((w.head * rows_of(D) + w.g) * (2 * D + 16) + 32 * w.t);
    const uint32_t f_at = smem_addr(buf.f_new + w.head * rows_of(D) + 2 * w.t);
    if (w.lane < rows_of(D)) buf.fr[w.warp * rows_of(D) + w.lane] = make_float2(buf.f[w.head * rows_of(D) + w.lane], 0.f);
    {
        float zeros[2 * NT];
#pragma unroll
        for (int k = 0; k < 2 * NT; ++k) zeros[k] = 0.f;
        s.set_sums(zeros);
    }
    __syncwarp();
    const uint32_t ring = smem_addr(buf.ring);
    bool scaled = false;                   // O holds values x v_down, no longer what codes and blocks' scales stand for
    auto scale_values = [&]() {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) s.o[j][i][c] *= a.v_scale;
        scaled = true;
    };
    for (int j = p.j0; j < p.j1; ++j) {
        if (alive) {
            alive = rdattn::warp_wait(&sh.full[at.stage], at.parity, &sh.abort, kWaitBudget);
            if (!alive && w.lane == 0) {
                sh.abort = 1;
                rd_flag(a.status, RD_DEV_TIMEOUT);
            }
        }
        const uint32_t k_at = ring + (uint32_t)(at.stage * 2 * a.half), v_at = k_at + (uint32_t)a.half;
        if (j < p.n_ctx) {
            const int first = w.split * 16 * TILES, valid = p.C - j * chunk - first;
            Rows<BITS> k_row, v_row;
            k_row.swizzled = v_row.swizzled = a.tiled;
            k_row.pitch = v_row.pitch = a.pitch;
            uint32_t off = (uint32_t)(first * a.pitch);
            k_row.first = v_row.first = 0;
            if (BITS == 8 && a.tiled) {    // boxes of 128 bytes of the heads' rows
                k_row.first = v_row.first = (uint32_t)(w.head * D % 128);
                off += (uint32_t)(w.head * D / 128 * chunk * 128);
            } else {
                off += (uint32_t)(w.head * rdquant::row_bytes(D, BITS));
            }
            k_row.base = k_at + off;
            v_row.base = v_at + off;
            // (two tiles at a time where the registers last: more products in flight)
            constexpr int MT = D == 64 && NT > 2 ? 1 : TILES;
#pragma unroll 1
            for (int x = 0; x < TILES; x += MT)
                if (valid > 16 * x) {
                    context_tiles<D, BITS, NT, MT>(a, w, s, k_row, v_row, q_at, min(16 * MT, valid - 16 * x));
                    k_row.base += (uint32_t)(16 * a.pitch);
                    v_row.base += (uint32_t)(16 * a.pitch);
                }
        } else {
            const int tile = j - p.n_ctx;
            if (!scaled) scale_values();
            if (tile % w.splits == w.split) {
                const uint32_t off = (uint32_t)(w.head * D * 2);
                draft_tile<D, BITS, NT>(a, w, p, s, k_at + off, v_at + off, q_at, f_at, tile * kDraftTile,
                                        min(kDraftTile, p.len - tile * kDraftTile));
            }
        }
        __syncwarp();
        if (w.lane == 0) rdtc::mbar_arrive(&sh.empty[at.stage]);
        at.next(a.stages);
    }
    if (!scaled) scale_values();
    float l[2 * NT], r[2 * NT];
    s.sums(l);
    over_lanes<NT, true>(l);
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) r[k] = s.reference(k);

    // ---- the warps of a head join their sums, the upper half of them into the lower
    for (int n = w.splits; n > 1;) {
        const int half = (n + 1) / 2;
        const bool gives = w.split >= half && w.split < n, takes = w.split < n - half;
        const int slot = (takes ? w.split : w.split - half) * a.heads + w.head;
        float fo[2 * NT];
#pragma unroll
        for (int i0 = 0; i0 < NT; i0 += 2) {
            if (gives) {
                if (i0 == 0) {
#pragma unroll
                    for (int k = 0; k < 2 * NT; ++k) buf.join_ml[(slot * 8 + k) * 32 + w.lane] = make_float2(s.none >> k & 1u ? -INFINITY : r[k], l[k]);
                }
#pragma unroll
                for (int i = i0; i < i0 + 2 && i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        buf.join[((slot * 2 + i - i0) * (D / 16) + j) * 32 + w.lane] =
                            make_float4(s.o[j][i][0], s.o[j][i][1], s.o[j][i][2], s.o[j][i][3]);
            }
            compute_sync<D>();
            if (takes) {
                if (i0 == 0) {
#pragma unroll
                    for (int k = 0; k < 2 * NT; ++k) {
                        const float2 ml = buf.join_ml[(slot * 8 + k) * 32 + w.lane];
                        const float mine = s.none >> k & 1u ? -INFINITY : r[k];
                        const float m = fmaxf(mine, ml.x), mu = m == -INFINITY ? 0.f : m;
                        const float f = fast_exp2(mine - mu);
                        fo[k] = fast_exp2(ml.x - mu);
                        r[k] = mu;
                        if (m != -INFINITY) s.none &= ~(1u << k);
                        l[k] = l[k] * f + ml.y * fo[k];
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            s.o[j][k / 2][k & 1] *= f;
                            s.o[j][k / 2][2 + (k & 1)] *= f;
                        }
                    }
                }
#pragma unroll
                for (int i = i0; i < i0 + 2 && i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const float4 v = buf.join[((slot * 2 + i - i0) * (D / 16) + j) * 32 + w.lane];
                        s.o[j][i][0] += v.x * fo[2 * i];
                        s.o[j][i][1] += v.y * fo[2 * i + 1];
                        s.o[j][i][2] += v.z * fo[2 * i];
                        s.o[j][i][3] += v.w * fo[2 * i + 1];
                    }
            }
            compute_sync<D>();
        }
        n = half;
    }
    if (w.split != 0) return;

    // ---- rows, or partials of a unit that the ranges cut
    const bool whole = p.j0 == 0 && p.j1 == p.n(a);
    const int h = p.hg * a.heads + w.head;
    const size_t slot = ((size_t)2 * blockIdx.x + (p.j0 == 0 ? 1 : 0)) * a.heads + w.head;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int at = 8 * i + 2 * w.t + e;
            if (at >= p.rows) continue;
            if (whole) {
                const float f = l[2 * i + e] == 0.f ? 0.f : a.v_up * (1.f / l[2 * i + e]);
                const int row = p.r0 + at;
                uint32_t u[D / 16];
#pragma unroll
                for (int j = 0; j < D / 16; ++j) u[j] = pack_bf16(s.o[j][i][e] * f, s.o[j][i][2 + e] * f);
                uint4* o = reinterpret_cast<uint4*>(
                    a.o + (((size_t)p.b * a.P + row / a.G) * a.Hq + (size_t)h * a.G + row % a.G) * D + D / 8 * w.g);
#pragma unroll
                for (int j = 0; j < D / 64; ++j) o[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
            } else {
                float4* o = reinterpret_cast<float4*>(a.part + (slot * rows_of(D) + at) * D + D / 8 * w.g);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    o[j] = make_float4(s.o[2 * j][i][e], s.o[2 * j][i][2 + e], s.o[2 * j + 1][i][e], s.o[2 * j + 1][i][2 + e]);
                if (w.g == 0) a.part_ml[slot * rows_of(D) + at] = make_float2(s.none >> (2 * i + e) & 1u ? -INFINITY : r[2 * i + e], l[2 * i + e]);
            }
        }
}

// The unit that this CTA's range begins and does not end, for the merge: and the CTA that has its last chunk.
__device__ __forceinline__ void describe(const Args& a, const Division& d)
{
    int4 unit = make_int4(-1, 0, 0, 0);
    Walk walk = Walk::over(a, d);
    Piece p;
    while (walk.next(a, p)) {
        if (p.j0 != 0 || p.j1 >= p.n(a)) continue;
        const Shape s = shape_of(a, p.b);
        const uint64_t last = walk.S + (uint64_t)p.unit * s.unit_cost(a) + a.unit_cost + (uint64_t)(p.n(a) - 1) * s.chunk_cost(a);
        unit = make_int4(p.b, p.unit, (int)d.of(last), 0);
    }
    if ((threadIdx.x & 31) == 0) a.desc[blockIdx.x] = unit;
}

template <int D, int BITS>
__global__ void __launch_bounds__(threads_of(D), 1) quant_attention_kernel(const __grid_constant__ Args a)
{
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ Shared sh;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5;
    const int splits = warps_of(D) / a.heads;
    Buffers buf;
    buf.ring = dyn;
    buf.q = reinterpret_cast<__half*>(dyn + (size_t)a.stages * 2 * a.half);
    buf.f = reinterpret_cast<float*>(buf.q + (size_t)a.heads * rows_of(D) * (D + 8));
    buf.f_new = buf.f + (size_t)a.heads * rows_of(D);
    buf.fr = reinterpret_cast<float2*>(buf.f_new + (size_t)a.heads * rows_of(D));
    buf.l = buf.fr + warps_of(D) * rows_of(D);
    buf.join = reinterpret_cast<float4*>(buf.l + warps_of(D) * (rows_of(D) / 8) * 32);
    buf.join_ml = reinterpret_cast<float2*>(buf.join + warps_of(D) / 2 * 2 * (D / 16) * 32);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMostStages; ++i) {
            rdtc::mbar_init(&sh.full[i], a.tiled ? 1 : 32 * kLoaders);
            rdtc::mbar_init(&sh.empty[i], warps_of(D));
        }
        rdtc::mbar_init(&sh.never, 1);
        rdtc::mbar_fence_init();
        sh.abort = sh.never_abort = 0;
    }
    const Division d = divide<threads_of(D)>(a, sh.division);               // (its barriers order the set-up too)
    __syncthreads();
    if (warp >= warps_of(D)) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(load_regs(D)));
        if (!a.tiled) load_rowwise<D, BITS>(a, sh, buf.ring, d);
        else if (warp == warps_of(D)) load_tiled<D, BITS>(a, sh, buf.ring, d);
        if (warp == warps_of(D)) describe(a, d);       // (now, so that its code is not fetched beside that of the first chunks)
        clear_rows<D>(a);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(compute_regs(D)));
    Place w;
    w.warp = warp;
    w.lane = threadIdx.x & 31;
    w.g = w.lane >> 2;
    w.t = w.lane & 3;
    w.head = warp % a.heads;
    w.split = warp / a.heads;
    w.splits = splits;
    bool alive = true;
    if (a.stall > 0) {                     // the test hook: a wait that runs out
        alive = rdattn::warp_wait(&sh.never, 0, &sh.abort, a.stall);
        if (w.lane == 0) {
            sh.abort = 1;
            rd_flag(a.status, RD_DEV_TIMEOUT);
        }
    }
    Walk walk = Walk::over(a, d);
    Piece p;
    Turn at = {0, 0};
    while (walk.next(a, p)) {
        const int tiles = (p.rows + 7) / 8;
        if (tiles == 1) piece<D, BITS, 1>(a, sh, buf, w, p, at, alive);
        else if (tiles == 2) piece<D, BITS, 2>(a, sh, buf, w, p, at, alive);
        else if (tiles == 3) piece<D, BITS, 3>(a, sh, buf, w, p, at, alive);
        else if constexpr (rows_of(D) > 24) piece<D, BITS, 4>(a, sh, buf, w, p, at, alive);
    }
}

// o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the pieces of a cut unit.  A warp takes a row of
// one head, so that a few units of many pieces (long contexts) keep as many warps busy as they have rows (with one CTA
// for a head's rows, two contexts of 40,000 with 32 rows a head spent 90 of 132 us here).
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) quant_merge_kernel(const Args a)
{
    constexpr int kCols = D / 4, kShares = 32 / kCols;     // D = 64: two halves of the pieces
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 unit = a.desc[blockIdx.x];
    const int first = blockIdx.x, last = unit.z;
    if (unit.x < 0 || unit.x >= a.B || last <= first || last >= (int)gridDim.x) return;
    const int len = a.lens[unit.x];
    if (len <= 0 || len > a.P) return;
    Shape s;
    s.len = len;
    const int groups = s.groups(a), hg = unit.y / groups, r0 = unit.y % groups * s.per(a);
    const int rows = min(s.per(a), s.rows(a) - r0), h = hg * a.heads + blockIdx.y, n = last - first + 1;
    const int lane = threadIdx.x & 31, c = lane % kCols, share = lane / kCols;
    for (int r = blockIdx.z * kMergeWarps + (threadIdx.x >> 5); r < rows; r += gridDim.z * kMergeWarps) {
        auto at = [&](int k) { return (((size_t)2 * (first + k) + (k == 0 ? 1 : 0)) * a.heads + blockIdx.y) * a.unit_rows + r; };
        float M = -INFINITY, L = 0.f;
        for (int k = lane; k < n; k += 32) M = fmaxf(M, a.part_ml[at(k)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float mu = M == -INFINITY ? 0.f : M;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < n; k0 += 32) {
            float f = 0.f;
            if (k0 + lane < n) {
                const float2 ml = a.part_ml[at(k0 + lane)];
                f = fast_exp2(ml.x - mu);
                L += f * ml.y;
            }
            const int some = min(32, n - k0);
            for (int k1 = 0; k1 < some; k1 += 8) {         // (eight pieces' loads under way together)
                float4 v[8 / kShares];
#pragma unroll
                for (int i = 0; i < 8 / kShares; ++i) {
                    const int k = k1 + i * kShares + share;
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < some) v[i] = reinterpret_cast<const float4*>(a.part)[at(k0 + k) * kCols + c];
                }
#pragma unroll
                for (int i = 0; i < 8 / kShares; ++i) {
                    const float by = __shfl_sync(0xffffffffu, f, k1 + i * kShares + share);      // (0 behind the last)
                    o.x += by * v[i].x, o.y += by * v[i].y, o.z += by * v[i].z, o.w += by * v[i].w;
                }
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        if constexpr (kShares == 2) {
            o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
        }
        const float f = L == 0.f ? 0.f : a.v_up * (1.f / L);
        const int row = r0 + r;
        if (share == 0) {
            uint2 out;
            out.x = pack_bf16(o.x * f, o.y * f);
            out.y = pack_bf16(o.z * f, o.w * f);
            reinterpret_cast<uint2*>(a.o)[((((size_t)unit.x * a.P + row / a.G) * a.Hq + (size_t)h * a.G + row % a.G) * D) / 4 + c] = out;
        }
    }
}

int heads_of(int Hkv) { return Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1; }

// bytes apart in shared memory: four rows that a half-warp reads at once start 8 banks apart (4
// bits), two that a quarter reads 16 banks (8 bits)
int pitch_of(int seg, int bits)
{
    const int step = bits == 4 ? 32 : 64;
    int p = (seg + step - 1) / step * step;
    if (p / step % 2 == 0) p += step;
    return p;
}

size_t desc_bytes(int grid) { return ((size_t)grid * sizeof(int4) + 127) & ~size_t(127); }

template <int D, int BITS>
cudaError_t launch(Args& a, int grid, cudaStream_t stream)
{
    const int chunk = 16 * tiles_of(D, BITS) * (warps_of(D) / a.heads);
    a.chunk = chunk;
    a.draft_chunk = kDraftTile;
    a.unit_rows = rows_of(D);
    a.row_step = 8;
    // (cycles of 64 positions x 4 heads, D = 128: 3,050 with 16 rows, 3,600 with 24, 4,700 with 32; a unit's
    // start and end 18,000.  Two contexts of 40,000 with 24 rows a head: 61 us with 120, 58 with 180, 55 with 240; 16 x 40 nodes
    // on 32/8 heads 86, 84 and 87.)
    a.chunk_cost = 16;
    a.step_cost = 5;
    a.unit_cost = 180 * 2 / tiles_of(D, BITS);              // (chunks of half the positions)
    a.least_cost = 72;
    a.seg = a.heads * rdquant::row_bytes(D, BITS);
    a.pitch = pitch_of(a.seg, BITS);
    const int stride = a.Hkv * rdquant::row_bytes(D, BITS);
    a.gran = a.seg % 16 == 0 && stride % 16 == 0 ? 16 : a.seg % 8 == 0 && stride % 8 == 0 ? 8 : 4;
    a.per_row = a.seg / a.gran;
    a.per_row_magic = (uint32_t)((0x100000000ULL + a.per_row - 1) / a.per_row);
    // TMA: rows of whole 16 bytes, the unit's part among them, and coordinates of 31 bits
    const int64_t rows_all = (int64_t)a.num_pages * a.page_size;
    a.tiled = a.gran == 16 && rows_all > 0 && rows_all <= 0x7fffffff && (BITS == 4 || a.seg % 128 == 0);
    if (a.tiled) {
        const int box = box_of(D, BITS), width = BITS == 4 ? a.seg : 128;
        if (!make_map(&a.k_map, a.k_pool, rows_all, stride, width, box, BITS == 8) ||
            !make_map(&a.v_map, a.v_pool, rows_all, stride, width, box, BITS == 8))
            return cudaErrorUnknown;
        a.pitch = width;
    }
    a.draft_pitch = a.heads * D * 2 + 16;
    const int rows = a.tiled ? chunk * a.seg : chunk * a.pitch, drafts = kDraftTile * a.draft_pitch;
    a.half = ((rows > drafts ? rows : drafts) + 1023) / 1024 * 1024;       // (swizzled tiles repeat every 1024 bytes)
    const int fixed = a.heads * rows_of(D) * ((D + 8) * 2 + 8) + warps_of(D) * (rows_of(D) + rows_of(D) / 8 * 32) * 8 + warps_of(D) / 2 * 32 * (2 * (D / 16) * 16 + 8 * 8);
    constexpr int kSmem = 227 * 1024 - 1024;               // what the static part leaves
    a.stages = (kSmem - fixed) / (2 * a.half);
    if (a.stages > kMostStages) a.stages = kMostStages;
    const int smem = a.stages * 2 * a.half + fixed;
    auto kernel = quant_attention_kernel<D, BITS>;
    static const cudaError_t ready = [&]() {
        cudaFuncAttributes f;
        cudaError_t e = cudaFuncGetAttributes(&f, kernel);
        // setmaxnreg deals out the registers of the launch
        return e != cudaSuccess ? e : f.numRegs == launch_regs(D) ? cudaSuccess : cudaErrorInvalidConfiguration;
    }();
    if (ready != cudaSuccess) return ready;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads_of(D), smem, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return cudaSuccess;
}

template <int D>
cudaError_t launch_merge(const Args& a, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    const long long rows = (long long)a.P * a.G < a.unit_rows ? (long long)a.P * a.G : a.unit_rows;
    cfg.gridDim = dim3((unsigned)grid, (unsigned)a.heads, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quant_merge_kernel<D>, a);
}

}  // namespace

size_t rd_quant_attention_workspace_bytes(int Hkv, int D)
{
    const int grid = rd_device_sm_count();
    const size_t rows = (size_t)2 * grid * heads_of(Hkv) * kMostRows;
    return desc_bytes(grid) + rows * (sizeof(float2) + (size_t)D * sizeof(float));
}

cudaError_t rd_launch_quant_attention(const rd_quant_kv& kv, int B, int P_max, int Hq, int Hkv, int D, float scale,
                                      const void* q, const void* k_new, const void* v_new, int max_ctx,
                                      const int32_t* packed_len, const uint32_t* mask, int mask_words, void* o,
                                      void* workspace, int32_t* dev_status, cudaStream_t stream)
{
    const int grid = rd_device_sm_count();
    Args a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k_new = static_cast<const __nv_bfloat16*>(k_new);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new);
    a.k_pool = static_cast<const unsigned char*>(kv.k_pool);
    a.v_pool = static_cast<const unsigned char*>(kv.v_pool);
    a.table = kv.pages.block_table;
    a.ctx_lens = kv.pages.ctx_lens;
    a.lens = packed_len;
    a.mask = mask;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.heads = heads_of(Hkv);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.desc = reinterpret_cast<int4*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + desc_bytes(grid));
    a.part = reinterpret_cast<float*>(a.part_ml + (size_t)2 * grid * a.heads * kMostRows);
    a.status = dev_status;
    a.B = B;
    a.P = P_max;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.mask_words = mask_words;
    a.num_pages = kv.pages.num_pages;
    a.page_size = kv.pages.page_size;
    a.max_pages = kv.pages.max_pages;
    // no context is longer than its row of the table, or there is no page to read
    const long long row = kv.pages.num_pages > 0 ? (long long)kv.pages.max_pages * kv.pages.page_size : 0;
    a.max_ctx = (int)(row < max_ctx ? row : max_ctx);
    int exponent;
    a.new_m = 2.f * (float)frexp(scale * kLog2e, &exponent);
    a.new_e = exponent - 1;
    a.ctx_m = 2.f * (float)frexp(scale * kLog2e * kv.k_scale, &exponent);
    a.ctx_e = exponent - 1;
    // (sums of 2^31 weights of up to 2^15 each, times values of up to 2688 v_scale, stay below 2^127)
    frexp(kv.v_scale, &exponent);
    a.v_up = ldexpf(1.f, exponent > 65 ? exponent - 65 : 0);
    a.v_down = 1.f / a.v_up;
    a.v_scale = kv.v_scale * a.v_down;
    a.stall = rd_attention_stall_budget();
    const cudaError_t e = D == 128 ? kv.bits == 4 ? launch<128, 4>(a, grid, stream) : launch<128, 8>(a, grid, stream)
                          : kv.bits == 4 ? launch<64, 4>(a, grid, stream)
                                         : launch<64, 8>(a, grid, stream);
    if (e != cudaSuccess) return e;
    return D == 128 ? launch_merge<128>(a, grid, stream) : launch_merge<64>(a, grid, stream);
}
