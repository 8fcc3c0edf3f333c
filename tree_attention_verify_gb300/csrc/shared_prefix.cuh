// What the kernels of rd_tree_attention_shared share: the plan in the workspace,
// the partials' layout, and the division of a chunk sequence over the CTAs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rd_internal.cuh"

namespace rdshared {

constexpr float kLog2e = 1.4426950408889634f;

// A group of requests, its live nodes in one compact list.
struct Group {
    int node0, nodes;      // its part of the list
    int positions;         // prefix length
    int leader;            // its first request with rows, whose table names the pages
    int unit0, pairs;      // its first unit, units (of 256 rows) per kv head
};

// What the plan kernel leaves in the workspace, and where the partials go: running
// maximum m (log2 units), sum l, and unnormalised O as float4 [D / 4][rows], so
// that a warp's accesses cover consecutive rows.
struct Plan {
    int32_t* eff_len;      // [B] packed length, 0: the request is skipped
    int32_t* skip;         // [B] prefix positions of the request
    int32_t* gid;          // [B] its group, -1: no prefix
    int32_t* node_base;    // [B + 1] its first node in the compact list
    int32_t* node_row;     // [B P_max] compact node -> b P_max + p
    Group* group;          // [n_groups]
    uint32_t* first;       // [n_groups + 1] what the groups before count in the prefix's division
    int4* req;             // [B] first unit of its group (-1: no prefix), units per kv head,
                           // first row within the group, first compact row
    // over the prefix: whole units by compact row, [Hkv][D / 4][rows_cap]; pieces of
    // units in slots, two per CTA, [slot][D / 4][256]
    int2* unit;            // [unit] pieces, and the first one's slot if several
    float4* rows;
    float2* rows_ml;
    size_t rows_cap;
    float4* part;
    float2* part_ml;
    // behind the prefix: the same, by row (b P_max + p) G + g, slots of slot_rows
    rd_shared_suffix suffix;
    float4* suf_part;
    float2* suf_part_ml;
    int slot_rows;
    int grid, suf_grid;    // CTAs of the two launches
    uint32_t* suf_first;   // [B + 1] suffix chunks of the requests before (shared_suffix.cu)
    int* suf_next;         // the next suffix unit that nobody has taken
};

// n CTAs of `grid` take the W chunks of a sequence in equal ranges, each of at least
// `least` chunks: CTA c starts at chunk floor(c W / n).
__device__ __forceinline__ uint32_t range_ctas(uint32_t W, uint32_t grid, uint32_t least)
{
    const uint32_t n = W / least;
    return n < 1u ? 1u : (n < grid ? n : grid);
}
__device__ __forceinline__ uint32_t range_start(uint32_t W, uint32_t n, uint32_t c)
{
    return (uint32_t)(((uint64_t)c * W) / n);
}
// the CTA whose range holds chunk x
__device__ __forceinline__ uint32_t range_of(uint32_t W, uint32_t n, uint32_t x)
{
    return (uint32_t)((((uint64_t)x + 1) * n - 1) / W);
}

constexpr int kUnitRows = 256;             // rows of a prefix unit

// The partials of one row: the first piece's, the others' (from slot to slot), and
// the distance between four-column groups.
struct Pieces {
    const float4* o0;
    const float2* ml0;
    const float4* o1;
    const float2* ml1;
    size_t o_step, ml_step, stride;
    int n;
    __device__ __forceinline__ const float4* o(int i) const { return i == 0 ? o0 : o1 + (size_t)(i - 1) * o_step; }
    __device__ __forceinline__ const float2* ml(int i) const { return i == 0 ? ml0 : ml1 + (size_t)(i - 1) * ml_step; }
};

// How many pieces an entry (pieces, first slot) of a table names, all in slots below
// 2 `grid`.  A launch whose waits ran out may have left an entry unwritten: what is
// no such entry counts as no pieces.
__device__ __forceinline__ int pieces_in(int2 unit, int grid)
{
    const bool fine = unit.x == 1 ||
                      (unit.x > 1 && unit.x <= grid && unit.y >= 0 && unit.y < 2 * grid && unit.y / 2 + unit.x <= grid);
    return fine ? unit.x : 0;
}

// unit = (pieces, first slot); a whole unit's rows are [h][D / 4][cap] at `row`,
// pieces lie in slots of R rows at r, those behind the first in slots 2 c
template <int D>
__device__ __forceinline__ Pieces pieces_at(int2 unit, const float4* rows, const float2* rows_ml, size_t cap, int h,
                                            size_t row, const float4* part, const float2* part_ml, int R, int r,
                                            int grid)
{
    Pieces p;
    p.n = pieces_in(unit, grid);
    if (p.n == 0) unit = make_int2(1, 0);
    const bool whole = unit.x == 1;
    const size_t next = 2 * (size_t)(unit.y / 2 + 1);
    p.stride = whole ? cap : (size_t)R;
    p.o0 = whole ? rows + (size_t)h * (D / 4) * cap + row : part + (size_t)unit.y * (D / 4) * R + r;
    p.ml0 = whole ? rows_ml + (size_t)h * cap + row : part_ml + (size_t)unit.y * R + r;
    p.o1 = part + next * (D / 4) * R + r;
    p.ml1 = part_ml + next * R + r;
    p.o_step = (size_t)2 * (D / 4) * R;
    p.ml_step = (size_t)2 * R;
    return p;
}

// the pieces over the prefix, of compact row `row`, row r of its unit
template <int D>
__device__ __forceinline__ Pieces pieces_of(int2 unit, const Plan& p, int h, int row, int r)
{
    return pieces_at<D>(unit, p.rows, p.rows_ml, p.rows_cap, h, (size_t)row, p.part, p.part_ml, kUnitRows, r, p.grid);
}

// ---- the suffix kernel for few rows per kv head (shared_suffix.cu)
constexpr int kSuffixRows = 64;            // of a unit at most
// nodes of a unit (all G heads of each)
__host__ __device__ constexpr int rd_suffix_nodes(int P_max, int G) { return P_max * G <= kSuffixRows ? P_max : kSuffixRows / G; }
// chunks per CTA at least: 1, 2 and 4 make 4 requests x 32 heads x 20 rows (10 of them
// live) 29.1, 28.3 and 30.8 us
constexpr uint32_t kSuffixMinChunks = 2;
// warps of 16 rows for `rows` rows
__host__ __device__ constexpr int rd_suffix_row_warps(int rows) { return (rows + 15) / 16; }
// positions of a chunk: with one or two row warps several warps split them
__host__ __device__ constexpr int rd_suffix_chunk(int row_warps) { return row_warps <= 2 ? 64 : 32; }
// CTAs per SM: what registers leave room for (a row warp's sums take half of its
// registers; five warps a CTA leave 168 each to two CTAs, 128 to three, which spills)
__host__ __device__ constexpr int rd_suffix_ctas(int row_warps) { return row_warps == 3 ? 3 : 2; }

// A launch that may start before its predecessor in the stream has ended.
inline cudaError_t launch_dependent(const void* kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                    void** args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace rdshared

int rd_suffix_grid(int rows);
bool rd_suffix_by_unit(long long units, int grid);
cudaError_t rd_launch_shared_suffix(const rdshared::Plan& p, int B, int P_max, int Hq, int Hkv, int D,
                                    float scale_log2, const void* q, const void* k_new, const void* v_new,
                                    const void* k_pool, const void* v_pool, const rd_paged_kv& paged,
                                    const uint32_t* mask, int mask_words, bool by_unit, void* o, int32_t* dev_status,
                                    cudaStream_t stream);
