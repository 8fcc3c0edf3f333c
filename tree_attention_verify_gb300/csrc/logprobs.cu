// rd_token_logprobs and rd_accepted_logprobs: for rows x of V logits, with p = softmax(x / T),
// log p(token), the entropy H = -sum p log p, and the k most likely tokens.
//
// One pass over each row.  In units of log2, with c = log2(e) / T and a reference m,
//   z = c (x - m),  l = sum 2^z,  w = sum 2^z z:
//   log p(x_t) = (x_t - m) / T - ln l,   H = ln l - ln 2 w / l.
// The reference is the maximum of the CTA's first 16,384 logits; a thread that meets a larger one
// moves its own.  So a logit costs a difference, a product, an exponential and two accumulations:
// about 50 instructions for eight 16-bit logits, somewhat more than half of what the SM can
// issue while HBM delivers them.  What is rare (a larger maximum, a candidate, numbers at the ends of
// the range) stays out of the loop's way.  4,096 rows of 128,256 bf16 logits with 20 alternatives
// take 223.5 us (4.7 TB/s; 40,000 instructions a row, whose loads' latency is not hidden all of the time).
//
// The top k come from the same pass: a threshold that at least k logits of the row reach
// is known after the first 64 logits of each thread (the k-th largest of the threads'
// maxima, found bit by bit); the 16-byte groups with what reaches it afterwards, a few times k of
// them, are kept, and their 64-bit keys (value, then the lower index first) ranked by counting at the end.  Where these
// overfill the list (many equal logits), its k-th key is a better threshold for another pass; where they do so again (a
// row that keeps rising), a threshold is searched in a few more (608 rising rows of 128,256 with 20 alternatives: 478 us,
// ordinary ones 41).
//
// Few rows: a cluster of up to eight CTAs takes one, and its first CTA joins the parts.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rd_internal.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 8;                  // 16-byte loads of a thread in flight
constexpr int kMostCtas = 8;               // of a row
constexpr int kList = 1024;                // candidates of a CTA
constexpr int kGroups = 512;               // 16-byte groups that hold some
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
    const void* logits;
    const int32_t* rows;                   // row of entry n (null: n)
    const int32_t* tokens;
    // the accepted path's rows, where `unpacker` is given: entry (b, i)
    const int32_t *unpacker, *best, *accepted;
    int W, L, P;
    int64_t n, rows_total;
    int V, k;
    // log2(e) / T, and what c is short of, relative; two numbers' difference over T is (a h - b h) / Th and
    // in units of log2 (a h - b h) ch, with h 1/2 where the difference may leave the range and its quotient not
    float c, off, h, Th, ch;
    float *logprob, *entropy;
    int32_t* top;
    float* top_logprob;
    int32_t* status;
};

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float exp2_(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two 32-bit numbers in one operation each
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 both(uint64_t x)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// ------------------------------------------------------------------ 16 bytes of logits
// The fast way takes logits below kLow as that, and references between -1e38 and 1e30: differences
// are finite, and those of such logits have no weight.  It sums 2^z (x - m), at most 150 / c each,
// and for c between 1e-27 and 1e27 2^30 of them stay within the range.
constexpr float kLow = -3.0e38f;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4])
    {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static constexpr uint32_t kNone = 0xff800000u;       // -inf
    // with what lies below kLow as that
    static __device__ __forceinline__ void unpack_finite(const uint4& u, float (&x)[4])
    {
        unpack(u, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = max_nan(x[i], kLow);
    }
    static __device__ __forceinline__ float top(const uint4& u)
    {
        return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)), max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ float one(const void* p, int64_t i)
    {
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
    }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ void unpack_finite(const uint4& u, float (&x)[8])
    {
        constexpr uint32_t low = 0xff62ff62u;            // kLow
        unpack(make_uint4(max2(u.x, low), max2(u.y, low), max2(u.z, low), max2(u.w, low)), x);
    }
    static __device__ __forceinline__ float top(const uint4& u)
    {
        const uint32_t t = max2(max2(u.x, u.y), max2(u.z, u.w));
        return max_nan(__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u));
    }
};
template <>
struct Vec<__half> {
    static constexpr int n = 8;
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return __half2float(static_cast<const __half*>(p)[i]); }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
    static constexpr uint32_t kNone = 0xfc00fc00u;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ void unpack_finite(const uint4& u, float (&x)[8])
    {
        unpack(u, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = max_nan(x[i], kLow);
    }
    static __device__ __forceinline__ float top(const uint4& u)
    {
        const uint32_t t = max2(max2(u.x, u.y), max2(u.z, u.w));
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&t));
        return max_nan(v.x, v.y);
    }
};

// numbers as unsigned ones of the same order (-0 as +0), and back
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float number(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ unsigned long long key_of(float x, int i)
{
    return (unsigned long long)ordered(x) << 32 | (uint32_t)~i;
}

// the difference of two logits in units of log2
struct Slope {
    float h, c;
    __device__ __forceinline__ float operator()(float a, float b) const { return (a * h - b * h) * c; }
};

struct Stats {
    // Reference (a logit; -inf: nothing yet), sums of the others, and how many stand at the reference: where one token has
    // nearly all of the probability, log l is that of 1 + l, and nothing of l is lost beside the 1.
    float m, l, w, ones;
    __device__ __forceinline__ void move(float to, Slope slope)   // to another reference
    {
        if (m != -INFINITY) {
            const float z = slope(m, to), f = exp2_(z), all = l + ones;
            w = f * (w + z * all);
            l = f * all;
            if (f == 0.f) w = 0.f;
        }
        ones = 0.f;
        m = to;
    }
    // (sums of 2^z and 2^z (x - m))
    __device__ __forceinline__ void add(float2 ls, float2 ws, float c) { l += ls.x + ls.y, w = fmaf(ws.x + ws.y, c, w); }
};

struct Shared {
    unsigned long long list[kList];
    uint4 group[kGroups];                  // groups in which some logit reaches the threshold, and their numbers
    int group_id[kGroups];
    int groups;
    unsigned long long best[32];           // this CTA's top k, in order
    unsigned long long from[kMostCtas][32];
    Stats part[kMostCtas];                 // of the CTAs of the cluster
    Stats warp[kWarps];
    int count;
    int digit, above, reach;               // of search()
};

__device__ __forceinline__ void push(Shared& sh, unsigned long long key)
{
    const int at = atomicAdd(&sh.count, 1);
    if (at < kList) sh.list[at] = key;
}

// The row's 16-byte groups (of aligned addresses: the first and the last may lie partly outside
// of it), and the share of this CTA.
template <typename T>
struct Row {
    static constexpr int N = Vec<T>::n;
    const T* x;
    const uint4* base;
    int V, off, first, last;               // elements of group 0 before the row; this CTA's groups
    __device__ __forceinline__ Row(const T* row, int V_, int part, int parts) : x(row), V(V_)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row);
        off = (int)((at & 15) / sizeof(T));
        base = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
        const int groups = (V + off + N - 1) / N, each = (groups + parts - 1) / parts;
        first = min(groups, part * each);
        last = min(groups, first + each);
    }
    __device__ __forceinline__ bool inside(int g) const { return g * N >= off && (g + 1) * N - off <= V; }
    __device__ __forceinline__ int index(int g, int e) const { return g * N + e - off; }
    // a group that lies partly outside of the row, element by element; what is outside counts as -inf
    __device__ __noinline__ uint4 edge(int g) const
    {
        union {
            uint4 u;
            T x[N];
        } v;
        constexpr uint32_t none = Vec<T>::kNone;
        v.u = make_uint4(none, none, none, none);
        for (int e = 0; e < N; ++e) {
            const int i = index(g, e);
            if (i >= 0 && i < V) v.x[e] = x[i];
        }
        return v.u;
    }
    __device__ __forceinline__ uint4 group(int g) const;
};

__device__ __forceinline__ uint4 load16(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename T>
__device__ __forceinline__ uint4 Row<T>::group(int g) const { return inside(g) ? load16(base + g) : edge(g); }

// a group that has a candidate
__device__ __forceinline__ void keep(Shared& sh, int g, const uint4& u)
{
    const int at = atomicAdd(&sh.groups, 1);
    if (at < kGroups) {
        sh.group[at] = u;
        sh.group_id[at] = g;
    }
}

// the logits of group g whose keys reach `least`
template <typename T>
__device__ __noinline__ void collect(Shared& sh, const Row<T>& row, int g, uint4 u, unsigned long long least)
{
    constexpr int N = Vec<T>::n;
    float x[N];
    Vec<T>::unpack(u, x);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int i = row.index(g, e);
        const unsigned long long key = key_of(x[e], i);
        if (key >= least && i >= 0 && i < row.V) push(sh, key);
    }
}

// One group after the other: the one with the reference itself, and all of rows where the fast way would not do
// (references near the lowest number, extreme temperatures).  2^-200 is 0, and 0 x -200 too: a logit of -inf
// adds nothing.
template <typename T>
__device__ __noinline__ Stats add_slowly(Stats s, uint4 u, float top, Slope slope)
{
    constexpr int N = Vec<T>::n;
    if (top == -INFINITY) return s;
    if (!(top <= s.m)) s.move(top, slope);
    float v[N];
    Vec<T>::unpack(u, v);
    for (int e = 0; e < N; ++e) {
        const float d = slope(v[e], s.m), z = max_nan(d, -200.f), p = exp2_(z);
        if (d == 0.f) {
            s.ones += 1.f;
        } else {
            s.l += p;
            s.w = fmaf(p, z, s.w);
        }
    }
    return s;
}

// One warp: sh.list[0 .. n) -> sh.best, the keys of rank below k, in order.  The bits of the k-th largest are found one by
// one until at most 64 keys reach them (the whole key's if need be: equal logits differ in their places), which
// are ranked by counting.
__device__ __forceinline__ void rank(Shared& sh, int n, int k)
{
    const int lane = threadIdx.x & 31;
    unsigned long long at = 0;
    int reached = n;
    for (unsigned long long bit = 1ull << 63; bit != 0 && reached > 64; bit >>= 1) {
        int reach = 0;
        for (int i = lane; i < n; i += 32) reach += sh.list[i] >= (at | bit);
        reach = __reduce_add_sync(0xffffffffu, reach);
        if (reach >= k) at |= bit, reached = reach;
    }
    unsigned long long* kept = reinterpret_cast<unsigned long long*>(sh.group);
    int m = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const unsigned long long key = i0 + lane < n ? sh.list[i0 + lane] : 0;
        const bool mine = i0 + lane < n && key >= at;
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (mine) kept[m + __popc(who & ((1u << lane) - 1))] = key;
        m += __popc(who);
    }
    sh.best[lane] = 0;
    __syncwarp();
    for (int i = lane; i < m; i += 32) {
        const unsigned long long key = kept[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) r += kept[j] > key;
        if (r < k) sh.best[r] = key;
    }
    __syncwarp();
}

// A lower bound of the row's k-th key that at most kList keys of this CTA's share (more than k) reach: eight of its bits in a
// pass over them, eight passes at most.
template <typename T>
__device__ __noinline__ unsigned long long search(Shared& sh, const Row<T>& row, int k)
{
    constexpr int N = Vec<T>::n;
    int* const counts = reinterpret_cast<int*>(sh.group);                  // of the 256 digits
    const int tid = threadIdx.x, lane = tid & 31;
    unsigned long long found = 0;          // the key's bits from `shift` up
    int above = 0;                         // keys that are larger in these bits
    for (int shift = 56;; shift -= 8) {
        static_assert(kThreads == 256, "a thread a digit");
        counts[tid] = 0;
        __syncthreads();
        for (int g0 = row.first; g0 < row.last; g0 += kThreads) {
            const int g = g0 + tid;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (g < row.last) u = row.group(g);
            float x[N];
            Vec<T>::unpack(u, x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int i = row.index(g, e);
                const unsigned long long key = key_of(x[e], i);
                const bool mine = g < row.last && i >= 0 && i < row.V && (shift == 56 || key >> (shift + 8) == found);
                const uint32_t who = __ballot_sync(0xffffffffu, mine);
                if (mine) {                // (most keys have one first digit: a lane adds for all of its warp that share it)
                    const int digit = (int)(key >> shift) & 255;
                    const uint32_t same = __match_any_sync(who, digit);
                    if (lane == __ffs(same) - 1) atomicAdd(&counts[digit], __popc(same));
                }
            }
        }
        __syncthreads();
        // the largest digit that k keys reach
        int reach = above;
        for (int d = 255; d > tid; --d) reach += counts[d];
        if (reach < k && reach + counts[tid] >= k) {
            sh.digit = tid;
            sh.above = reach;
            sh.reach = reach + counts[tid];
        }
        __syncthreads();
        found = found << 8 | (unsigned long long)sh.digit;
        above = sh.above;
        const int reached = sh.reach;
        __syncthreads();                   // (all have read them)
        if (reached <= kList || shift == 0) return found << shift;
    }
}

// the sums of a warp's lanes, in all of them
__device__ __forceinline__ Stats join_warp(Stats s, Slope slope)
{
    const float m = number(__reduce_max_sync(0xffffffffu, ordered(s.m)));
    if (s.m != m) s.move(m, slope);            // (two equal references may be infinite)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.l += __shfl_xor_sync(0xffffffffu, s.l, o);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
        s.ones += __shfl_xor_sync(0xffffffffu, s.ones, o);
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ Args a)
{
    __shared__ Shared sh;
    constexpr int N = Vec<T>::n;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x / parts;
    const int k = a.k;

    // ---- the entry's row and token (the same for the whole cluster)
    int64_t r = n;
    int token = a.tokens[n];
    bool live = token != -1;
    unsigned wrong = 0;
    if (a.unpacker != nullptr) {
        const int b = (int)(n / a.L), i = (int)(n % a.L);
        const int w = a.best[b], acc = a.accepted[b];
        if (w < 0 || w >= a.W || acc < 0 || acc >= a.L) wrong = RD_DEV_BAD_INDEX;
        else if (i > acc) live = false;
        else {
            const int node = a.unpacker[((size_t)b * a.W + w) * a.L + i];
            if (node < 0 || node >= a.P) wrong = RD_DEV_BAD_INDEX;
            r = (int64_t)b * a.P + node;
        }
    } else if (a.rows != nullptr) {
        r = a.rows[n];
    }
    if (live && !wrong) {
        if (token < 0 || token >= a.V) wrong = RD_DEV_BAD_TOKEN;
        else if (r < 0 || r >= a.rows_total) wrong = RD_DEV_BAD_INDEX;
    }
    if (!live || wrong) {
        if (part == 0) {
            if (tid == 0) {
                if (wrong) rd_flag(a.status, wrong);
                a.logprob[n] = 0.f;
                a.entropy[n] = 0.f;
            }
            if (tid < k) {
                a.top[n * k + tid] = -1;
                a.top_logprob[n * k + tid] = 0.f;
            }
        }
        return;
    }
    // every CTA of the cluster has started before one writes into another's shared memory
    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    const T* x = static_cast<const T*>(a.logits) + r * a.V;
    const Row<T> row(x, a.V, part, parts);
    const float chosen = part == 0 && tid == 0 ? Vec<T>::one(x, token) : 0.f;
    if (tid == 0) sh.count = sh.groups = 0;
    Stats s = {-INFINITY, 0.f, 0.f, 0.f};
    uint64_t l2 = 0, w2 = 0;               // (two chains of sums each, of the reference s.m)
    const Slope slope = {a.h, a.ch};
    const uint64_t c2 = pair(a.c, a.c);
    unsigned long long least = 0;
    float floor_ = -INFINITY;              // what reaches it is looked at
    bool fast = false;                     // (where it is not, every group is looked at)
    constexpr int kStep = kThreads * kAhead;
    // groups that lie inside of the row: the first and the last of all may not
    const int inside0 = row.first + (row.first < row.last && !row.inside(row.first) ? 1 : 0);
    const int inside1 = row.last - (row.last > inside0 && !row.inside(row.last - 1) ? 1 : 0);
    // (a row without such a group comes to the counts below with no barrier on its way)
    if (inside0 >= inside1) __syncthreads();
    for (int g0 = inside0; g0 < inside1; g0 += kStep) {
        uint4 u[kAhead];
        if (g0 + kStep <= inside1) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) u[j] = load16(row.base + g0 + j * kThreads + tid);
        } else {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int g = g0 + j * kThreads + tid;
                u[j] = make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
                if (g < inside1) u[j] = load16(row.base + g);
            }
        }
        if (g0 == inside0) {
            float top = Vec<T>::top(u[0]);
#pragma unroll
            for (int j = 1; j < kAhead; ++j) top = max_nan(top, Vec<T>::top(u[j]));
            const uint32_t mine = g0 + tid < inside1 ? ordered(top) : 0u;
            const uint32_t warp_top = __reduce_max_sync(0xffffffffu, mine);
            if (lane == 0) sh.warp[warp].m = __uint_as_float(warp_top);
            __syncthreads();
            uint32_t most = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) most = max(most, __float_as_uint(sh.warp[w].m));
            s.m = number(most);
            floor_ = s.m;
            fast = s.m > -1e38f && s.m < 1e30f && a.c > 1e-27f && a.c < 1e27f;
            if (k > 0) {
                // the k-th largest of the threads' maxima, rounded down to 16 bits
                uint32_t at = 0;
                for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1)
                    if (__syncthreads_count(mine >> 16 >= (at | bit)) >= k) at |= bit;
                least = (unsigned long long)at << 48;
                floor_ = number(at << 16);
                if (at == 0 || floor_ != floor_) floor_ = -INFINITY;
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float top = Vec<T>::top(u[j]);
            if (!(top < floor_)) {
                const int g = g0 + j * kThreads + tid;
                if (k > 0 && g < inside1) keep(sh, g, u[j]);
                if (fast && !(top < s.m)) {
                    if (top != s.m) {
                        s.add(both(l2), both(w2), a.c);
                        l2 = w2 = 0;
                        fast = top < 1e30f;
                    }
                    s = add_slowly<T>(s, u[j], top, slope);
                    continue;
                }
            }
            if (!fast) {
                s = add_slowly<T>(s, u[j], top, slope);
                continue;
            }
            float v[N];
            Vec<T>::unpack_finite(u[j], v);
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const uint64_t d = add2(pair(v[e], v[e + 1]), pair(-s.m, -s.m));
                const float2 z = both(mul2(d, c2));
                const uint64_t p = pair(exp2_(z.x), exp2_(z.y));
                l2 = add2(l2, p);
                w2 = fma2(p, d, w2);
            }
        }
    }
    s.add(both(l2), both(w2), a.c);
    // the row's first and last group, where they are partly outside
    if (tid < 2) {
        const int g = tid == 0 ? row.first : row.last - 1;
        if (tid == 0 ? inside0 > row.first : inside1 < row.last) {
            const uint4 u = row.edge(g);
            const float top = Vec<T>::top(u);
            if (k > 0 && !(top < floor_)) keep(sh, g, u);
            s = add_slowly<T>(s, u, top, slope);
        }
    }
    __syncthreads();                       // (sh.warp is read above and written below; the groups are there)
    if (k > 0 && sh.groups <= kGroups)
        for (int i = tid; i < sh.groups; i += kThreads) collect<T>(sh, row, sh.group_id[i], sh.group[i], least);
    s = join_warp(s, slope);
    if (lane == 0) sh.warp[warp] = s;
    __syncthreads();
    if (k > 0) {
        // Too many: the k-th of those kept is a better threshold for another pass.  Where that is not enough either (a
        // row that keeps rising, whose first keys tell nothing of the last), the threshold is searched.
        bool again = sh.groups > kGroups;
        for (int pass = 0; again || sh.count > kList; ++pass) {
            if (pass == 0) {
                if (again) {
                    // (of the groups that were kept, if the keys are not yet a list)
                    for (int i = tid; i < kList / N; i += kThreads) collect<T>(sh, row, sh.group_id[i], sh.group[i], least);
                    __syncthreads();
                }
                if (warp == 0) rank(sh, min(sh.count, kList), k);
                __syncthreads();
                least = max(least, sh.best[k - 1]);
            } else {
                least = search<T>(sh, row, k);
            }
            again = false;
            floor_ = number((uint32_t)(least >> 32));
            if (floor_ != floor_) floor_ = -INFINITY;
            __syncthreads();
            if (tid == 0) sh.count = 0;
            __syncthreads();
            for (int g = row.first + tid; g < row.last; g += kThreads) {
                const uint4 u = row.group(g);
                if (!(Vec<T>::top(u) < floor_)) collect<T>(sh, row, g, u, least);
            }
            __syncthreads();
        }
        if (warp == 0) rank(sh, sh.count, k);
    }
    Stats all = {-INFINITY, 0.f, 0.f, 0.f};     // (in the first warp)
    if (warp == 0) {
        if (lane < kWarps) all = sh.warp[lane];
        all = join_warp(all, slope);
    }
    if (parts > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        Shared* to = cluster.map_shared_rank(&sh, 0);
        if (tid < 32) to->from[part][tid] = sh.best[tid];
        if (tid == 0) to->part[part] = all;
        cluster.sync();
        if (part != 0) return;
        if (warp == 0) {
            all = {-INFINITY, 0.f, 0.f, 0.f};
            if (lane < parts) all = sh.part[lane];
            all = join_warp(all, slope);
        }
        if (k > 0) {
            // at most 8 x 32 keys, one a thread
            const unsigned long long key = tid < parts * 32 ? sh.from[tid / 32][lane] : 0;
            if (tid < 32) sh.best[tid] = 0;
            __syncthreads();
            if (key != 0) {
                int rk = 0;
                for (int p = 0; p < parts; ++p)
                    for (int j = 0; j < k; ++j) rk += sh.from[p][j] > key;
                if (rk < k) sh.best[rk] = key;
            }
            __syncthreads();
        }
    }
    const float l = all.l + all.ones, mean = kLn2 * (all.w / l);          // of (x - m) / T
    const float ln_l = all.ones > 0.f ? logf(all.ones) + log1pf(all.l / all.ones) : logf(l);
    // A c that is off by `off` moves log l by as much of the mean: for log p, whose difference is over T itself, it is given back.
    const float ln_p = fmaf(a.off, mean, ln_l);
    const float m = all.m == -INFINITY ? 0.f : all.m;
    if (tid == 0) {
        a.logprob[n] = (chosen * a.h - m * a.h) / a.Th - ln_p;
        a.entropy[n] = ln_l - mean;
    }
    if (tid < k) {
        const unsigned long long key = sh.best[tid];
        a.top[n * k + tid] = (int32_t)~(uint32_t)key;
        a.top_logprob[n * k + tid] = (number((uint32_t)(key >> 32)) * a.h - m * a.h) / a.Th - ln_p;
    }
}

template <typename T>
cudaError_t launch(const Args& a, cudaStream_t stream)
{
    // a row on several CTAs while they all run at once and each has a few thousand logits
    const int sms = rd_device_sm_count();
    int parts = 1;
    while (parts < kMostCtas && a.n * parts * 2 <= 2 * sms && a.V / (parts * 2) >= 2048) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a);
}

}  // namespace

cudaError_t rd_launch_logprobs(const rd_logprobs& q, cudaStream_t stream)
{
    Args a = {};
    a.logits = q.logits;
    a.rows = q.rows;
    a.tokens = q.tokens;
    a.unpacker = q.unpacker;
    a.best = q.best_beam;
    a.accepted = q.n_accepted;
    a.W = q.W;
    a.L = q.L;
    a.P = q.P_max;
    a.n = q.n;
    a.rows_total = q.n_rows;
    a.V = q.V;
    a.k = q.top;
    const double c = 1.4426950408889634 / q.temperature;
    a.c = (float)c;
    a.off = (float)((c - a.c) / c);
    a.h = q.temperature > 1.f ? 0.5f : 1.f;
    a.Th = q.temperature * a.h;
    a.ch = a.c / a.h;
    a.logprob = q.logprob;
    a.entropy = q.entropy;
    a.top = q.top_tokens;
    a.top_logprob = q.top_logprobs;
    a.status = q.dev_status;
    if (q.dt == RD_BF16) return launch<__nv_bfloat16>(a, stream);
    if (q.dt == RD_F16) return launch<__half>(a, stream);
    return launch<float>(a, stream);
}
