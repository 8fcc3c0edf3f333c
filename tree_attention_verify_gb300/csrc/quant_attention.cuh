// rd_tree_attention_quant's arguments, the division of its work among the CTAs, and small loads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "quant_format.cuh"
#include "rd_internal.cuh"

namespace rdquant {

using rdattn::fast_exp2;
using rdattn::pack_bf16;
using rdtc::smem_addr;

constexpr long long kWaitBudget = 4000000000LL;     // cycles, about two seconds
constexpr double kLog2e = 1.4426950408889634;
// A row's weights are powers of two above a reference that lies kBelow under the row's maximum,
// or up to kLag more: a weight P reaches 2^15 (a 16-bit float ends at 2^16), O is
// rescaled only when the reference lags more, and weights down to 2^-21 of the largest
// keep all 11 bits, those below an absolute 2^-32 of it.
constexpr float kBelow = 7.f, kLag = 8.f;

struct Args {
    const __nv_bfloat16 *q, *k_new, *v_new;
    const unsigned char *k_pool, *v_pool;
    const int32_t *table, *ctx_lens, *lens;
    const uint32_t* mask;
    __nv_bfloat16* o;
    float* part;               // [2 grid slots][heads][unit_rows][D]
    float2* part_ml;           // [2 grid slots][heads][unit_rows] reference (log2 units), sum
    int4* desc;                // [grid] the unit that a CTA begins and does not end
    int32_t* status;
    int B, P, Hq, Hkv, G, mask_words, num_pages, page_size, max_pages, max_ctx;
    // Scores in log2 units: of cached keys product x ctx_m 2^ctx_e (the cache's scale in it), of drafts x new_m 2^new_e.
    float ctx_m, new_m;
    int ctx_e, new_e;
    // O holds values x v_down, a power of two that keeps sums of values up to the largest numbers finite
    float v_scale, v_down, v_up;       // the cache's scale x v_down; 1 / v_down
    long long stall;
    int heads;                 // kv heads of a unit
    int unit_rows, row_step;   // rows of a unit at most, a multiple of row_step
    int chunk, draft_chunk;    // positions, packed drafts of a chunk
    uint32_t chunk_cost, step_cost, unit_cost, least_cost;     // see Shape
    int seg, pitch, gran, per_row;     // bytes of a position's rows, apart in shared memory, a copy; copies
    uint32_t per_row_magic;
    int draft_pitch, half, stages;     // bytes of a stage's K (and of its V)
    bool tiled;                // the pools' rows come as TMA boxes
    CUtensorMap k_map, v_map;
};

// ------------------------------------------------------------------ the division of the work
// A unit is (request, group of `heads` kv heads, group of up to `unit_rows` rows).  Its chunks
// (context, then tiles of drafts) stand in one sequence with all other units', weighted by what
// they cost, and the CTAs take equal ranges of it.  Widening a chunk costs the same for any number
// of rows (chunk_cost), its products go with them (step_cost for each row_step rows); a unit's start and
// end take as long as a few chunks (unit_cost).  A range is at least least_cost, more than any
// chunk.  (A unit of 2^31 positions in chunks of 32 costs less than 2^32.)
struct Shape {
    int len, C;                // nodes (0: the request is skipped or has none), context
    __device__ __forceinline__ int rows(const Args& a) const { return len * a.G; }
    // row groups, and rows of a group
    __device__ __forceinline__ int groups(const Args& a) const { return (rows(a) + a.unit_rows - 1) / a.unit_rows; }
    __device__ __forceinline__ int per(const Args& a) const
    {
        return ((rows(a) + groups(a) - 1) / groups(a) + a.row_step - 1) & ~(a.row_step - 1);
    }
    // chunks of the context, and all
    __device__ __forceinline__ int n_ctx(const Args& a) const
    {
        return (int)(((uint32_t)C + (uint32_t)a.chunk - 1u) / (uint32_t)a.chunk);
    }
    __device__ __forceinline__ int n(const Args& a) const { return n_ctx(a) + (len + a.draft_chunk - 1) / a.draft_chunk; }
    __device__ __forceinline__ uint32_t chunk_cost(const Args& a) const
    {
        return a.chunk_cost + a.step_cost * (uint32_t)(per(a) / a.row_step);
    }
    __device__ __forceinline__ uint32_t unit_cost(const Args& a) const { return a.unit_cost + (uint32_t)n(a) * chunk_cost(a); }
    __device__ __forceinline__ uint64_t cost(const Args& a) const
    {
        return len == 0 ? 0 : (uint64_t)unit_cost(a) * (uint32_t)(groups(a) * (a.Hkv / a.heads));
    }
};

__device__ __forceinline__ Shape shape_of(const Args& a, int b)
{
    Shape s;
    s.len = a.lens[b];
    s.C = 0;
    if (s.len <= 0 || s.len > a.P) {
        s.len = 0;
        return s;
    }
    s.C = a.ctx_lens[b];
    if (s.C < 0 || s.C > a.max_ctx) s.len = 0;
    return s;
}

struct Division {
    uint64_t W;                // cost of everything
    uint32_t n;                // CTAs that work
    int b;                     // the request in which this CTA's range begins
    uint64_t S;                // cost of the requests before it
    uint64_t each;             // floor(W / n): the first W mod n ranges have one more
    uint32_t rest;
    __device__ __forceinline__ uint64_t begin(uint32_t c) const { return each * c + min(c, rest); }
    __device__ __forceinline__ uint32_t of(uint64_t x) const      // the CTA whose range holds x
    {
        uint32_t lo = 0, hi = n;
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if (begin(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

struct Piece {
    int b, unit;               // request, unit within it
    int hg, r0, rows;          // head group, first row, rows
    int j0, j1;                // chunks of this piece
    int C, len, n_ctx;         // context, nodes, chunks of the context
    __device__ __forceinline__ int n(const Args& a) const { return n_ctx + (len + a.draft_chunk - 1) / a.draft_chunk; }
};

// The pieces of a CTA's range, one after the other; every warp walks through them by itself.
struct Walk {
    uint64_t lo, hi, S;        // the range, and where the request begins
    int b, unit;               // the next unit to look at (-1: the first in the range)
    static __device__ __forceinline__ Walk over(const Args& a, const Division& d)
    {
        const uint32_t c = blockIdx.x;
        const bool idle = d.W == 0 || c >= d.n;
        Walk w;
        w.S = d.S;
        w.b = idle ? a.B : d.b;
        w.unit = -1;
        w.lo = idle ? 0 : d.begin(c);
        w.hi = idle ? 0 : c + 1 < d.n ? d.begin(c + 1) : d.W;
        return w;
    }
    __device__ __forceinline__ bool next(const Args& a, Piece& p)
    {
        while (b < a.B && S < hi) {
            const Shape s = shape_of(a, b);
            if (s.len != 0) {
                const uint32_t uc = s.unit_cost(a), c = s.chunk_cost(a);
                const int groups = s.groups(a), units = groups * (a.Hkv / a.heads);
                if (unit < 0) {
                    unit = 0;
                    if (lo > S) {          // (lo - S) / uc, below 2^22, from a quotient that is off by one at most
                        const uint64_t x = lo - S;
                        unit = (int)__fdividef((float)x, (float)uc);
                        if ((uint64_t)unit * uc > x) --unit;
                        else if ((uint64_t)(unit + 1) * uc <= x) ++unit;
                    }
                }
                while (unit < units) {
                    const uint64_t at = S + (uint64_t)unit * uc, first = at + a.unit_cost;
                    if (at >= hi) return false;
                    const int n = s.n(a);
                    // (a range that ends behind the unit takes all of its chunks)
                    const uint32_t j0 = lo > first ? (uint32_t)min((uint64_t)uc, lo - first) : 0;
                    const uint32_t j1 = hi > first ? (uint32_t)min((uint64_t)uc, hi - first) : 0;
                    p.j0 = (int)((j0 + c - 1) / c);
                    p.j1 = min(n, (int)((j1 + c - 1) / c));
                    p.unit = unit++;
                    if (p.j0 >= p.j1) continue;
                    p.b = b;
                    p.hg = p.unit / groups;
                    p.r0 = p.unit % groups * s.per(a);
                    p.rows = min(s.per(a), s.rows(a) - p.r0);
                    p.C = s.C;
                    p.len = s.len;
                    p.n_ctx = s.n_ctx(a);
                    return true;
                }
                S += s.cost(a);
            }
            unit = 0;
            ++b;
        }
        return false;
    }
};

// Shared memory of the division.
struct DivisionShared {
    int b;
    unsigned long long S, sum[32];
};

// Every CTA sums the requests' costs and finds the request where its range begins.
template <int kThreads>
__device__ __forceinline__ Division divide(const Args& a, DivisionShared& sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long mine = 0;
    for (int b = tid; b < a.B; b += kThreads) {
        const Shape s = shape_of(a, b);
        mine += s.cost(a);
        if (blockIdx.x == 0 && s.len != a.lens[b]) rd_flag(a.status, RD_DEV_BAD_LENGTH);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh.sum[warp] = mine;
    __syncthreads();
    Division d;
    d.W = 0;
    for (int w = 0; w < kThreads / 32; ++w) d.W += sh.sum[w];
    d.n = gridDim.x;
    if (d.W < (uint64_t)gridDim.x * a.least_cost) d.n = max(1u, (uint32_t)d.W / a.least_cost);
    d.each = d.W / d.n;
    d.rest = (uint32_t)(d.W - d.each * d.n);
    d.b = a.B;
    d.S = 0;
    __syncthreads();
    if (d.W == 0 || blockIdx.x >= d.n) return d;
    const uint64_t lo = d.begin(blockIdx.x);
    uint64_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        const unsigned long long cost = b < a.B ? shape_of(a, b).cost(a) : 0;
        unsigned long long inc = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sh.sum[warp] = inc;
        if (tid == 0) sh.b = -1;
        __syncthreads();
        uint64_t base = before;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) base += sh.sum[w];
            before += sh.sum[w];
        }
        const uint64_t S = base + inc - cost;
        if (cost != 0 && S <= lo && lo < S + cost) {
            sh.b = b;
            sh.S = S;
        }
        __syncthreads();
        const int found = sh.b;
        const uint64_t at = sh.S;
        __syncthreads();
        if (found >= 0) {
            d.b = found;
            d.S = at;
            break;
        }
    }
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
// where the 64 positions from pos0 + 64 k of request b lie: the pool's row
__device__ __forceinline__ int64_t row_at(const Args& a, int b, int pos, bool flags)
{
    int page = a.table[(size_t)b * a.max_pages + pos / a.page_size];
    if (page < 0 || page >= a.num_pages) {
        if (flags) rd_flag(a.status, RD_DEV_BAD_INDEX);
        page = 0;
    }
    return (int64_t)page * a.page_size + pos % a.page_size;
}

// ------------------------------------------------------------------ host side
// the pool as [rows][row bytes]; boxes of `box` rows x `width` bytes
inline bool make_map(CUtensorMap* map, const void* pool, int64_t rows, int row_bytes, int width, int box, bool swizzled)
{
    auto fn = rdattn::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)row_bytes / 4, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t boxes[2] = {(cuuint32_t)width / 4, (cuuint32_t)box};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(pool), dims, strides, boxes, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace rdquant
