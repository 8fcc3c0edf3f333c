// What writes the quantised paged cache and reads it back (formats in quant_format.cuh):
// rd_append_quant (prompts), rd_commit_accepted_quant (the accepted path of a step),
// rd_read_quant.
//
// In 4 bits a block of 16 elements x has the scale s = e4m3(min(448, amax |x| / (6 g))) and the
// codes e2m1(x / (g s)), ties to the even code, saturating; 0 where s is 0.  In 8 bits the codes
// are e4m3(x / g), saturating.
//
// All three are streams, bound by HBM: a thread takes one block of K and the same of V
// (32 bytes each on the 16-bit side, one access; 9 or 16 on the other), so that a block's maximum needs
// no other thread and neighbours' accesses are consecutive.  A CTA first finds where each of its
// tokens lies (request, position, page: a search and two dependent reads), a thread per token, then
// moves about kBlocks blocks.  Codes are the nearest to the exact quotients: by products with a reciprocal, and by the sign
// of an exact remainder where a border between two codes is within their error (about one value in 250,000, and those
// of few bits).  IEEE divisions, whose rounded quotients hide on which side of a border they are, also took longer (12,000
// tokens written and read back: 39 us, not 34).
// Two 16-byte accesses for a block's 32 bytes would take longer (16 x 4,096 tokens of 8 heads read from 4
// bits: 53 us, not 45), and so would CTAs of 1,024 blocks, which wait longer for their first
// bytes than they then move (the same: 39 us, not 37, with the divisions).  Reading 8 x 8,192 tokens of 40 heads
// from 8 bits takes 234 us, 6.9 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "quant_format.cuh"
#include "rd_internal.cuh"

namespace {

using namespace rdquant;

constexpr int kThreads = 256;
constexpr int kBlocks = 512;               // blocks of 16 elements that a CTA moves (of K, and of V)
constexpr int kMostTokens = 64;            // tokens of a CTA

// A tensor's scale: g, and m / (up1 up2) with m in [1, 2) and powers of two; inv is 1 / m in 8 bits, 1 / (6 m) in 4.
// A value times up1, then up2 over m is x / g whatever g is: up1 and up2 lie on one side of 1, so what leaves the
// range on the way saturates or is 0 anyway.
struct Scale {
    float g, m, up1, up2, inv;
    uint32_t last;             // 1 where g has more than nine bits
};

struct Pools {
    unsigned char *k, *v;
    Scale k_scale, v_scale;
    int num_pages, page_size, max_pages;
    const int32_t* table;
};

// the pool's row for position `pos` of table row b, or -1 (flagged)
__device__ __forceinline__ int64_t row_of(const Pools& p, int b, int64_t pos, int32_t* status)
{
    const int64_t slot = pos / p.page_size;
    if (slot >= p.max_pages) {
        rd_flag(status, RD_DEV_BAD_LENGTH);
        return -1;
    }
    const int page = p.table[(size_t)b * p.max_pages + slot];
    if (page < 0 || page >= p.num_pages) {
        rd_flag(status, RD_DEV_BAD_INDEX);
        return -1;
    }
    return (int64_t)page * p.page_size + pos % p.page_size;
}

// the last of n ascending offsets that is not above t (0 if all are)
template <typename T>
__device__ __forceinline__ int request_of(const T* __restrict__ offsets, int n, int64_t t)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if ((int64_t)offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------------ one block
__device__ __forceinline__ void unpack16(const uint32_t (&u)[8], float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// The code nearest to a quotient a / d is decided by an approximation y of it (products with a reciprocal, at most
// 3 units of its last place off), unless a border between two codes is as near.  Borders have BITS bits behind the
// first one at most: `apart` is at most 8 where some number of so few bits lies within 4 units.
template <int BITS>
__device__ __forceinline__ uint32_t apart(float y)
{
    return (__float_as_uint(y) + 4u) & ((1u << (23 - BITS)) - 1u);
}
// Such a y on the right side of the border t, or t itself: by the sign of |a| - t (d + e), which two fused
// operations give exactly (t d has few bits more than a 32-bit number, and nearly all cancel).
template <int BITS>
__device__ __forceinline__ float settled(float y, float a, float d, float e)
{
    const uint32_t u = __float_as_uint(fabsf(y)), t = (u + (1u << (22 - BITS))) & ~((1u << (23 - BITS)) - 1u);
    const float border = __uint_as_float(t), r = fmaf(-border, e, fmaf(-border, d, fabsf(a)));
    return apart<BITS>(fabsf(y)) > 8u ? y : copysignf(__uint_as_float(r > 0.f ? t + 8u : r < 0.f && t != 0 ? t - 8u : t), y);
}

__device__ __forceinline__ uint32_t e4m3_of(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t e2m1_of(const float* x)        // eight codes
{
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, e};\n\t}"
        : "=r"(d)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return d;
}

__device__ __forceinline__ float scale_value(uint32_t byte)
{
    uint32_t lo, hi;
    e4m3x4(byte, lo, hi);
    return __half2float(__ushort_as_half((unsigned short)lo));
}

template <int D, int BITS>
__device__ __forceinline__ void store_block(unsigned char* row, int block, const float (&x)[16], const Scale& g)
{
    const auto scaled = [&](float v) { return v * g.up1 * g.up2; };      // v / g = scaled(v) / m
    float y[16];
    if constexpr (BITS == 8) {
        uint32_t near = 9;
        const float by = g.up2 * g.inv;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y[i] = x[i] * g.up1 * by;
            near = min(near, apart<4>(y[i]));
        }
        if (near <= 8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = settled<4>(y[i], scaled(x[i]), g.m, 0.f);
        }
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = e4m3_of(y[4 * i], y[4 * i + 1]) | e4m3_of(y[4 * i + 2], y[4 * i + 3]) << 16;
        *reinterpret_cast<uint4*>(row + 16 * block) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
        float quotient = top * g.up1 * (g.up2 * g.inv);
        if (apart<4>(quotient) <= 8) {
            const float d = 6.f * g.m;
            quotient = settled<4>(quotient, scaled(top), d, fmaf(6.f, g.m, -d));
        }
        const uint32_t byte = e4m3_of(fminf(448.f, quotient), 0.f) & 0xffu;
        const float s = scale_value(byte), d = s * g.m;
        uint32_t u[2] = {0, 0};
        if (s > 0.f) {
            uint32_t near = 9;
            const float by = g.up2 * (1.f / d);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y[i] = x[i] * g.up1 * by;
                near = min(near, apart<2>(y[i]));
            }
            if (near <= 8) {
                const float e = fmaf(s, g.m, -d);
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = settled<2>(y[i], scaled(x[i]), d, e);
            }
            u[0] = e2m1_of(y);
            u[1] = e2m1_of(y + 8);
        }
        uint32_t* to = reinterpret_cast<uint32_t*>(row + 8 * block);
        if constexpr (D == 128) {
            *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);      // rows of 72 bytes
        } else {
            to[0] = u[0];                                                // of 36
            to[1] = u[1];
        }
        row[D / 2 + block] = (unsigned char)byte;
    }
}

// v g as a number of 32 bits that rounds to 16 bits as the exact product does: cut off, with its last bit set.  A product
// midway between two 16-bit numbers has nine bits at most, and so has g then, which divides it; with such a g every
// product fits and its last bit stays.
__device__ __forceinline__ float product(float v, const Scale& g)
{
    return __uint_as_float(__float_as_uint(__fmul_rz(v, g.g)) | g.last);
}

// a block as it lies in the pool, and its values
template <int D, int BITS>
struct Raw {
    uint4 c;                               // 4 bits: codes, codes, scale
    __device__ __forceinline__ void load(const unsigned char* row, int block)
    {
        if constexpr (BITS == 8) {
            c = __ldg(reinterpret_cast<const uint4*>(row + 16 * block));
        } else {
            if constexpr (D == 128) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + 8 * block));
                c.x = u.x, c.y = u.y;
            } else {
                const uint32_t* from = reinterpret_cast<const uint32_t*>(row + 8 * block);
                c.x = __ldg(from), c.y = __ldg(from + 1);
            }
            c.z = __ldg(row + D / 2 + block);
        }
    }
    __device__ __forceinline__ void values(const Scale& g, uint32_t (&o)[8]) const
    {
        uint32_t w[8];                     // 16-bit floats, in order
        if constexpr (BITS == 8) {
            e4m3x4(c.x, w[0], w[1]);
            e4m3x4(c.y, w[2], w[3]);
            e4m3x4(c.z, w[4], w[5]);
            e4m3x4(c.w, w[6], w[7]);
        } else {
            uint32_t s, same, u[4];
            e4m3x4(c.z * 0x01010101u, s, same);
            e2m1x8(c.x, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = mul_f16x2(u[i], s);          // exact
            e2m1x8(c.y, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 + i] = mul_f16x2(u[i], s);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<__half2*>(&w[i]));
            __nv_bfloat162 r = __floats2bfloat162_rn(product(v.x, g), product(v.y, g));
            o[i] = *reinterpret_cast<uint32_t*>(&r);
        }
    }
};

// 32 bytes in one access, where they are aligned so
__device__ __forceinline__ void store32(uint4* to, const uint32_t (&o)[8], bool aligned)
{
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}
__device__ __forceinline__ void load32(const uint4* from, uint32_t (&o)[8], bool aligned)
{
    if (aligned) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                     : "l"(from));
    } else {
        const uint4 a = __ldg(from), b = __ldg(from + 1);
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    }
}
__device__ __forceinline__ bool aligned32(const void* a, const void* b)
{
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 31) == 0;
}

// ------------------------------------------------------------------ writing
struct Where {
    int64_t from, to;                      // row of the source, of the pool (-1: none)
};

// tokens of the prompts: row t of [T, Hkv, D] belongs to the sequence of cu_seqlens that holds t
struct Prompt {
    static constexpr bool kSearched = true;
    const int32_t *cu, *ctx;
    int32_t* new_ctx;
    int B;
    int64_t T;
    __device__ __forceinline__ bool fine(int b) const
    {
        const int from = cu[b], to = cu[b + 1], C = ctx[b];
        return from >= 0 && from <= to && to <= T && C >= 0 && C <= 0x7fffffff - (to - from);
    }
    __device__ __forceinline__ void lengths(int i, int32_t* status) const
    {
        if (i >= B) return;
        const bool ok = fine(i);
        if (!ok) rd_flag(status, RD_DEV_BAD_LENGTH);
        new_ctx[i] = ctx[i] + (ok ? cu[i + 1] - cu[i] : 0);
    }
    // Whether request i has tokens that the search finds elsewhere, or nowhere: where cu does not ascend.  The search comes
    // to i from the tokens between the entries that it passes on its way.
    __device__ __forceinline__ bool lost(int i) const
    {
        if (i >= B || !fine(i) || cu[i] == cu[i + 1]) return false;
        int lo = 0, hi = B;
        bool found = true;
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (i >= mid) found &= cu[i] >= cu[mid], lo = mid;
            else found &= cu[i + 1] <= cu[mid], hi = mid;
        }
        return !found;
    }
    __device__ __forceinline__ Where find(const Pools& p, int64_t t, int32_t* status) const
    {
        const int b = request_of(cu, B, t);
        if (t < cu[b] || t >= cu[b + 1] || !fine(b)) return {t, -1};
        return at(p, b, t, status);
    }
    __device__ __forceinline__ Where at(const Pools& p, int b, int64_t t, int32_t* status) const
    {
        return {t, row_of(p, b, (int64_t)ctx[b] + (t - cu[b]), status)};
    }
};

// the accepted path: token t is position t % L of request t / L
struct Accepted {
    static constexpr bool kSearched = false;
    const int32_t *unpacker, *best, *accepted, *ctx;
    int32_t* new_ctx;
    int B, W, L, P;
    // how many tokens request b appends (0: its inputs are wrong)
    __device__ __forceinline__ int count(int b, unsigned& wrong) const
    {
        const int w = best[b], n = accepted[b], C = ctx[b];
        wrong = 0;
        if (w < 0 || w >= W || n < 0 || n >= L || C < 0) wrong = RD_DEV_BAD_INDEX;
        else if (C > 0x7fffffff - n - 1) wrong = RD_DEV_BAD_LENGTH;       // the new length leaves 31 bits
        return wrong ? 0 : n + 1;
    }
    __device__ __forceinline__ void lengths(int i, int32_t* status) const
    {
        if (i >= B) return;
        unsigned wrong;
        const int n = count(i, wrong);
        if (wrong) rd_flag(status, wrong);
        new_ctx[i] = ctx[i] + n;
    }
    __device__ __forceinline__ Where find(const Pools& p, int64_t t, int32_t* status) const
    {
        const int b = (int)(t / L), i = (int)(t % L);
        unsigned wrong;
        if (i >= count(b, wrong)) return {0, -1};
        const int64_t to = row_of(p, b, (int64_t)ctx[b] + i, status);
        const int node = unpacker[((size_t)b * W + best[b]) * L + i];
        if (to >= 0 && (node < 0 || node >= P)) {
            rd_flag(status, RD_DEV_BAD_INDEX);
            return {0, -1};
        }
        return {(int64_t)b * P + node, to};
    }
};

template <int D, int BITS, class Source>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ Source src, const __grid_constant__ Pools p,
                                                         int64_t tokens, int each, int Hkv, const uint4* __restrict__ k,
                                                         const uint4* __restrict__ v, int32_t* status)
{
    __shared__ Where where[kMostTokens];
    bool lost = false;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < src.B; i += (int64_t)gridDim.x * kThreads) {
        src.lengths((int)i, status);
        if constexpr (Source::kSearched) lost |= src.lost((int)i);
    }
    const int64_t t0 = (int64_t)blockIdx.x * each;
    int n = (int)min((int64_t)each, tokens - t0);
    if ((int)threadIdx.x < n) where[threadIdx.x] = src.find(p, t0 + threadIdx.x, status);
    lost = __syncthreads_or(lost);
    const int blocks = Hkv * (D / 16);     // of a token
    const bool wide = aligned32(k, v);
    int64_t q = 0;
    int done = 0;
    for (;;) {
        for (int i = threadIdx.x; i < n * blocks; i += kThreads) {
            const int t = i / blocks, c = i - t * blocks;
            const Where at = where[t];
            if (at.to < 0) continue;
            const size_t from = ((size_t)at.from * blocks + c) * 2;
            uint32_t ku[8], vu[8];
            load32(k + from, ku, wide);
            load32(v + from, vu, wide);
            const size_t to = ((size_t)at.to * Hkv + c / (D / 16)) * row_bytes(D, BITS);
            float x[16];
            unpack16(ku, x);
            store_block<D, BITS>(p.k + to, c % (D / 16), x, p.k_scale);
            unpack16(vu, x);
            store_block<D, BITS>(p.v + to, c % (D / 16), x, p.v_scale);
        }
        if (!Source::kSearched || !lost) return;
        // Sequences that do not ascend: the q-th request of those whose lengths this CTA has written, if its search
        // misses any of its tokens, whole, some tokens at a time (what is written twice are the same bytes).
        if constexpr (Source::kSearched) {
            int64_t b;
            for (;; ++q, done = 0) {
                b = (q / kThreads * gridDim.x + blockIdx.x) * kThreads + q % kThreads;
                if (b >= src.B) return;
                if (src.lost((int)b) && done < src.cu[b + 1] - src.cu[b]) break;
            }
            __syncthreads();
            n = min(kMostTokens, src.cu[b + 1] - src.cu[b] - done);
            if ((int)threadIdx.x < n) where[threadIdx.x] = src.at(p, (int)b, (int64_t)src.cu[b] + done + threadIdx.x, status);
            done += n;
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ reading
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Pools p, const int64_t* __restrict__ offsets,
                                                        const int32_t* __restrict__ starts, int B, int64_t total, int each,
                                                        int Hkv, uint4* __restrict__ k, uint4* __restrict__ v,
                                                        int32_t* status)
{
    __shared__ int64_t where[kMostTokens];             // the pool's row; -1: zeros; -2: not of any request
    const int64_t t0 = (int64_t)blockIdx.x * each;
    const int n = (int)min((int64_t)each, total - t0);
    if ((int)threadIdx.x < n) {
        const int64_t t = t0 + threadIdx.x;
        const int b = request_of(offsets, B, t);
        const int64_t from = offsets[b], to = offsets[b + 1], start = starts != nullptr ? starts[b] : 0;
        int64_t row = -2;
        if (t >= from && t < to) {
            if (from < 0 || to > total || start < 0) {
                rd_flag(status, RD_DEV_BAD_LENGTH);
                row = -1;
            } else {
                row = row_of(p, b, start + (t - from), status);
            }
        }
        where[threadIdx.x] = row;
    }
    if (blockIdx.x == 0)                               // offsets that do not ascend, or leave the output
        for (int b = threadIdx.x; b < B; b += kThreads)
            if (offsets[b] < 0 || offsets[b] > offsets[b + 1] || offsets[b + 1] > total) rd_flag(status, RD_DEV_BAD_LENGTH);
    __syncthreads();
    const int blocks = Hkv * (D / 16);
    const bool wide = aligned32(k, v);
    for (int i = threadIdx.x; i < n * blocks; i += kThreads) {
        const int t = i / blocks, c = i - t * blocks;
        const int64_t row = where[t];
        if (row == -2) continue;
        uint32_t ku[8] = {}, vu[8] = {};
        if (row >= 0) {
            const size_t from = ((size_t)row * Hkv + c / (D / 16)) * row_bytes(D, BITS);
            Raw<D, BITS> kr, vr;
            kr.load(p.k + from, c % (D / 16));
            vr.load(p.v + from, c % (D / 16));
            kr.values(p.k_scale, ku);
            vr.values(p.v_scale, vu);
        }
        const size_t to = ((size_t)(t0 + t) * blocks + c) * 2;
        store32(k + to, ku, wide);
        store32(v + to, vu, wide);
    }
}

int tokens_of_cta(int Hkv, int D)
{
    const int n = kBlocks / (Hkv * (D / 16));
    return n < 1 ? 1 : n > kMostTokens ? kMostTokens : n;
}

Scale scale_of(float g, int bits)
{
    int e;
    Scale s;
    s.g = g;
    s.m = 2.f * frexpf(g, &e);
    s.inv = 1.f / (bits == 8 ? s.m : 6.f * s.m);
    s.last = s.m * 256.f != truncf(s.m * 256.f);
    s.up1 = ldexpf(1.f, (1 - e) / 2);
    s.up2 = ldexpf(1.f, (1 - e) - (1 - e) / 2);
    return s;
}

Pools pools_of(const rd_quant_kv& kv)
{
    Pools p;
    p.k = static_cast<unsigned char*>(kv.k_pool);
    p.v = static_cast<unsigned char*>(kv.v_pool);
    p.k_scale = scale_of(kv.k_scale, kv.bits);
    p.v_scale = scale_of(kv.v_scale, kv.bits);
    p.num_pages = kv.pages.num_pages;
    p.page_size = kv.pages.page_size;
    p.max_pages = kv.pages.max_pages;
    p.table = kv.pages.block_table;
    return p;
}

template <int D, int BITS, class Source>
cudaError_t launch_write(const Source& src, const rd_quant_kv& kv, int64_t tokens, int Hkv, const void* k, const void* v,
                         int32_t* status, cudaStream_t stream)
{
    const int each = tokens_of_cta(Hkv, D);
    const int64_t ctas = tokens > 0 ? (tokens + each - 1) / each : 1;     // one for the lengths alone
    write_kernel<D, BITS, Source><<<(unsigned)ctas, kThreads, 0, stream>>>(
        src, pools_of(kv), tokens, each, Hkv, static_cast<const uint4*>(k), static_cast<const uint4*>(v), status);
    return cudaGetLastError();
}

template <class Source>
cudaError_t write(const Source& src, const rd_quant_kv& kv, int64_t tokens, int Hkv, int D, const void* k, const void* v,
                  int32_t* status, cudaStream_t stream)
{
    if (D == 128)
        return kv.bits == 4 ? launch_write<128, 4>(src, kv, tokens, Hkv, k, v, status, stream)
                            : launch_write<128, 8>(src, kv, tokens, Hkv, k, v, status, stream);
    return kv.bits == 4 ? launch_write<64, 4>(src, kv, tokens, Hkv, k, v, status, stream)
                        : launch_write<64, 8>(src, kv, tokens, Hkv, k, v, status, stream);
}

template <int D, int BITS>
cudaError_t launch_read(const rd_quant_kv& kv, const int64_t* offsets, const int32_t* starts, int B, int64_t total, int Hkv,
                        void* k, void* v, int32_t* status, cudaStream_t stream)
{
    const int each = tokens_of_cta(Hkv, D);
    read_kernel<D, BITS><<<(unsigned)((total + each - 1) / each), kThreads, 0, stream>>>(
        pools_of(kv), offsets, starts, B, total, each, Hkv, static_cast<uint4*>(k), static_cast<uint4*>(v), status);
    return cudaGetLastError();
}

}  // namespace

int64_t rd_quant_tokens_most(int Hkv, int D) { return (int64_t)0x7fffffff * tokens_of_cta(Hkv, D); }

cudaError_t rd_launch_append_quant(const rd_quant_kv& kv, int B, int Hkv, int D, const void* k, const void* v, int64_t total,
                                   const int32_t* cu_seqlens, const int32_t* ctx_lens, int32_t* new_ctx_lens,
                                   int32_t* dev_status, cudaStream_t stream)
{
    Prompt src;
    src.cu = cu_seqlens;
    src.ctx = ctx_lens;
    src.new_ctx = new_ctx_lens;
    src.B = B;
    src.T = total;
    return write(src, kv, total, Hkv, D, k, v, dev_status, stream);
}

cudaError_t rd_launch_commit_quant(const rd_quant_kv& kv, int B, int W, int L, int P_max, int Hkv, int D, const void* k_new,
                                   const void* v_new, const int32_t* unpacker, const int32_t* best_beam,
                                   const int32_t* n_accepted, const int32_t* ctx_lens, int32_t* new_ctx_lens,
                                   int32_t* dev_status, cudaStream_t stream)
{
    Accepted src;
    src.unpacker = unpacker;
    src.best = best_beam;
    src.accepted = n_accepted;
    src.ctx = ctx_lens;
    src.new_ctx = new_ctx_lens;
    src.B = B;
    src.W = W;
    src.L = L;
    src.P = P_max;
    return write(src, kv, (int64_t)B * L, Hkv, D, k_new, v_new, dev_status, stream);
}

cudaError_t rd_launch_read_quant(const rd_quant_kv& kv, int B, int Hkv, int D, const int64_t* offsets, const int32_t* starts,
                                 int64_t total, void* k_out, void* v_out, int32_t* dev_status, cudaStream_t stream)
{
    if (D == 128)
        return kv.bits == 4 ? launch_read<128, 4>(kv, offsets, starts, B, total, Hkv, k_out, v_out, dev_status, stream)
                            : launch_read<128, 8>(kv, offsets, starts, B, total, Hkv, k_out, v_out, dev_status, stream);
    return kv.bits == 4 ? launch_read<64, 4>(kv, offsets, starts, B, total, Hkv, k_out, v_out, dev_status, stream)
                        : launch_read<64, 8>(kv, offsets, starts, B, total, Hkv, k_out, v_out, dev_status, stream);
}
