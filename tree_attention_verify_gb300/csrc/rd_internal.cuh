// Internal helpers shared by the librd kernels (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rd.h"

#define RD_WARP 32

// OR error bits into the caller's device status word; never traps.
__device__ __forceinline__ void rd_flag(int32_t* status, unsigned bits)
{
    if (status != nullptr) atomicOr(reinterpret_cast<int*>(status), static_cast<int>(bits));
}

// Number of SMs of the current device (looked up once per device); the grid
// and split plans are sized from it.  Without a visible device (a host-only
// workspace query) it returns kRdFallbackSms, the count of a GB300.
constexpr int kRdFallbackSms = 152;
int rd_device_sm_count();

// Clock budget of the planted wait armed by rd_debug_stall_attention (0 = off).
long long rd_attention_stall_budget();

// Longest context of a request over pages: the kernels round it up to whole chunks in 32 bits.
constexpr int kRdMaxContext = 0x7fffffff - 256;

// Launchers (one per kernel family), called by the C entry points in rd_api.cu
// after host-side validation.  Each returns the cudaGetLastError() of its launches.
cudaError_t rd_launch_pack(const int32_t* beams, int B, int W, int L, int P_cap,
                           int32_t* tokens, int32_t* packer, int32_t* unpacker,
                           uint32_t* mask, int32_t* depth, int32_t* packed_len,
                           int32_t* dev_status, cudaStream_t stream);

cudaError_t rd_launch_unpack(const void* packed, int esize, int B, int P_max, int Dh,
                             const int32_t* unpacker, int W, int L, void* out,
                             int32_t* dev_status, cudaStream_t stream);

struct rd_accept_plan {
    int splits;        // vocab chunks per packed row
    int chunk;         // elements per chunk (multiple of 8)
};
rd_accept_plan rd_accept_make_plan(int B, int P_max, int V);
size_t rd_accept_workspace_bytes(int B, int P_max);
cudaError_t rd_launch_greedy_accept(const void* logits, int B, int P_max, int V,
                                    const int32_t* beams, const int32_t* unpacker,
                                    const int32_t* packed_len, int W, int L,
                                    int32_t* argmax, int32_t* accept_len,
                                    int32_t* best_beam, int32_t* n_accepted,
                                    int32_t* out_tokens, void* workspace,
                                    int32_t* dev_status, cudaStream_t stream);

cudaError_t rd_launch_sample_accept(const void* target, const void* draft, int B, int P_max,
                                    int V, float temperature, const int32_t* beams,
                                    const int32_t* packer, const int32_t* unpacker,
                                    const int32_t* packed_len, int W, int L,
                                    const float* u_accept, const float* u_sample,
                                    int32_t* accept_len, int32_t* best_beam,
                                    int32_t* n_accepted, int32_t* out_tokens,
                                    int32_t* dev_status, cudaStream_t stream);

// Tree attention (attention_tc.cu): the 16-bit, paged and FP8 variants.
struct rd_attn_plan {
    int tiles;         // row tiles per (request, kv head)
    bool stream_k;     // chunk-range division (tree attention), else whole units round-robin
    int grid;          // CTAs of the launch
    size_t ws_bytes;   // workspace bytes needed (chunk ranges: partials of cut units)
};
struct rd_paged_kv {
    const int32_t* block_table;   // [B, max_pages]
    const int32_t* ctx_lens;      // [B]
    int max_pages, page_size, num_pages;
};
struct rd_fp8_kv {
    const void* k_cache;          // e4m3 [total_ctx, Hkv, D]
    const void* v_cache;
    float k_scale, v_scale;
};
// The part of a shared-prefix call behind the prefix (shared_prefix.cu): fp32
// partials (running maximum m in log2 units, sum l, unnormalised O) instead of
// outputs, those of pieces in the workspace's slots.
struct rd_shared_suffix {
    const int32_t* skip;     // [B] positions that the group's prefix covers
    float4* rows;            // whole units: [Hkv][D / 4][rows_cap], row (b P_max + p) G + g
    float2* rows_ml;         // [Hkv][rows_cap]
    size_t rows_cap;         // B P_max G
    int2* unit;              // chunk ranges: [tile][b][kv head] pieces, first one's slot
};
rd_attn_plan rd_attn_make_plan(int B, int P_max, int Hq, int Hkv, int D, int max_kv);
cudaError_t rd_launch_attention(const rd_attn_plan& plan, int B, int P_max,
                                int Hq, int Hkv, int D, float scale, const void* q,
                                const void* k_new, const void* v_new,
                                const void* k_cache, const void* v_cache,
                                const int64_t* ctx_offsets, int64_t total_kv, int max_kv,
                                const int32_t* lens, const uint32_t* mask, int mask_words,
                                void* o, void* workspace, int32_t* dev_status,
                                cudaStream_t stream, const rd_paged_kv* paged = nullptr,
                                const rd_fp8_kv* fp8 = nullptr,
                                const rd_shared_suffix* shared = nullptr);

// Causal prefill with paired 128-row query tiles, one CTA per SM (causal_pair.cu).
cudaError_t rd_launch_causal_pair(int B, int Hq, int Hkv, int D, float scale, const void* q,
                                  const void* k, const void* v, const int32_t* cu_seqlens,
                                  int64_t total, int max_len, void* o, int32_t* dev_status,
                                  cudaStream_t stream);

cudaError_t rd_launch_commit(int B, int W, int L, int P_max, int Hkv, int D, const void* k_new,
                             const void* v_new, const int32_t* unpacker,
                             const int32_t* best_beam, const int32_t* n_accepted, void* k_pool,
                             void* v_pool, int num_pages, int page_size,
                             const int32_t* block_table, int max_pages, const int32_t* ctx_lens,
                             int32_t* new_ctx_lens, int32_t* dev_status, cudaStream_t stream);

cudaError_t rd_launch_beam_step(const void* logits, const float* scores_in,
                                const int32_t* beams_in, int B, int W, int V, int t,
                                int32_t* beams_out, float* scores_out, int32_t* parent,
                                int32_t* dev_status, cudaStream_t stream);

// Tree attention of groups that share a prefix (shared_prefix.cu).
// whether the part behind the prefix counts its work in 31 bits
bool rd_shared_suffix_counts(int B, int P_max, int Hq, int Hkv, int D, int max_ctx);
size_t rd_shared_workspace_bytes(int B, int P_max, int Hq, int Hkv, int D, int max_ctx, int n_groups);
cudaError_t rd_launch_shared_attention(int B, int P_max, int Hq, int Hkv, int D, float scale, const void* q,
                                       const void* k_new, const void* v_new, const void* k_pool,
                                       const void* v_pool, const rd_paged_kv& paged, int max_ctx,
                                       int n_groups, const int32_t* group_offsets,
                                       const int32_t* prefix_pages, const int32_t* packed_len,
                                       const uint32_t* mask, int mask_words, void* o, void* workspace,
                                       int32_t* dev_status, cudaStream_t stream);

// Page operators of the paged cache (pages.cu).
struct rd_page_pools {
    void* k_pool;             // [layers, num_pages, page_bytes]
    void* v_pool;
    int layers, num_pages;
    size_t page_bytes;
};
// small calls need no workspace
bool rd_fork_copies_itself(int n, int layers, size_t page_bytes);
bool rd_copy_resolves_itself(int n);
cudaError_t rd_launch_resize_pages(int32_t* block_table, int R, int max_pages, int32_t* row_pages,
                                   int32_t* page_refs, int num_pages, const int32_t* new_lens, int page_size,
                                   int32_t* dev_status, cudaStream_t stream);
cudaError_t rd_launch_fork_pages(const rd_page_pools& pools, int page_size, int32_t* block_table, int R,
                                 int max_pages, int32_t* row_pages, int32_t* page_refs, int32_t* ctx_lens,
                                 const int32_t* parent, const int32_t* child, int n, void* workspace,
                                 int32_t* dev_status, cudaStream_t stream);
cudaError_t rd_launch_copy_pages(const rd_page_pools& pools, const int32_t* src, const int32_t* dst, int n,
                                 void* workspace, int32_t* dev_status, cudaStream_t stream);
cudaError_t rd_launch_compact_pages(const rd_page_pools& pools, int32_t* block_table, int R, int max_pages,
                                    const int32_t* row_pages, int32_t* page_refs, int32_t* remap,
                                    int32_t* n_live, void* workspace, int32_t* dev_status, cudaStream_t stream);
