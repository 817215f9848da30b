// wq_logprobs.cu -- log probabilities of given tokens, the entropy and the k
// most likely alternatives of rows of logits, in one pass over the logits:
//
//     lse  = max_n x[n] + log sum_n exp(x[n] - max)
//     logprob[t] = x[t] - lse
//     entropy    = -sum_n p[n] log p[n] = log S - W / S,
//                  S = sum_n exp(x[n] - max),  W = sum_n exp(x[n] - max) (x[n] - max)
//     alternatives: the k largest x[n], ties to the lower index, as x[n] - lse
//
// Both terms of the entropy are positive (W <= 0, S >= 1), so it does not
// cancel.  A thread keeps a running maximum with its S and W and rescales them
// when the maximum grows, so the sums read every logit once (the alternatives read
// a few again) and nothing is written but the answers.
//
// Bound: HBM, 2 or 4 bytes per logit.  At that rate an SM has to take 12
// 16-bit logits a clock, three quarters of what its exponential unit can do
// and half of its issue slots, so the two sums run as packed fp32 pairs.
//
// Work split: a row goes to a cluster of C CTAs (1, 2, 4 or 8), each with one
// contiguous slice of it, whose answers meet through distributed shared
// memory: no workspace, no second launch, and one decode row still draws on
// eight SMs.  A CTA reads its slice in batches of kUnroll 16-byte vectors per
// thread, the next batch's loads in flight while it works on this one.
//
// Alternatives: the loop over the logits does nothing for them.  Behind it every
// thread knows the largest of the logits it read; a value that the maxima of at
// least k threads reach (and of few more: a search with one block-wide count a
// step) is reached by at least k logits, and only those threads' logits can be
// among the k largest; of those, the runs of vectors whose largest (kept in shared
// memory, at most 32 a thread) reaches it.  They are read again, by all threads
// together, and what reaches the value is kept and ranked.  Where much of the row
// shares the value (a mask that leaves fewer logits than alternatives) only what is
// above it is read again, and of the logits equal to it the first in the row, by a
// scan that ends with them.  Where more reaches it than the list holds all the same
// (rows of few distinct values) the k-th largest value is found by counting over
// those vectors.  A logit is ranked by a 64-bit key (value, then the complement of
// its index), so all keys differ and the answer is unique.
// (Collecting during the loop, against a bound raised as it went, took 307 us
// for 2048 rows of 152064 logits and k = 5.)
//
// Measured on B200, back to back in a graph: 2048 rows of 152064 bf16 logits 114 us
// without alternatives (5.5 TB/s), 118 with 5 and 135 with 64 (168 with 5 where a mask
// leaves a few logits a row); one such row with 20 alternatives 8.6; 77 rows of 50001
// fp32 logits with 64 15.5.  One call at a time from cold caches the 2048 rows take 133
// with 5.
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "wq.h"
#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int kUnroll = 4;     // 16-byte vectors per thread and batch
constexpr int kSortMax = 192;  // candidates ranked by counting without a cut first
constexpr int kListMax = 1024; // candidates of a CTA
constexpr int kChosenMax = 1024; // runs of vectors read again
constexpr int kRuns = 32;      // runs of a thread, at most
constexpr int kLpMaxCluster = 8;
constexpr int kShortBatches = 4; // rows of at most this many batches of a 128-thread CTA go to one

typedef unsigned long long key_t64;

struct LpParams {
    const void *logits;
    long long ld;
    int M, N, k, C, slice; // slice: elements per CTA, a multiple of the vector
    int run_batches;       // batches of a run
    const int32_t *tokens;
    float *logprob, *entropy, *top;
    int32_t *top_idx;
};

// Threads (or candidates) that a bound for k may let through where it can.
__host__ __device__ constexpr int lp_accept(int k) { return k + k / 2 + 8; }
static_assert(lp_accept(kTopkMaxK) <= kSortMax, "a cut list can be ranked");

// ---- packed fp32 pairs ----
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b),
                          z = *reinterpret_cast<unsigned long long *>(&c);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&r);
}

constexpr float kFarBelow = -200.f; // exp(-200) is 0 in fp32: masked and far logits add nothing, and 0 * -inf never forms

__device__ __forceinline__ float2 cut2(float2 d) // NaN stays NaN
{
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d.x) : "f"(kFarBelow));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d.y) : "f"(kFarBelow));
    return d;
}

// Far below m, and by a margin that 16-bit formats resolve whatever m is.
__device__ __forceinline__ float far_below(float m) { return m + kFarBelow - 0.02f * fabsf(m); }

template <class T>
struct LpType;
template <>
struct LpType<__nv_bfloat16> {
    static constexpr int VE = 8;
    // A pair's differences from the maximum m, far ones cut short: the pair is
    // held above `floor`, a pair far enough below m that what is cut counts for
    // nothing, which costs one instruction.  There is such a value from
    // m >= kFloorFrom on.
    static constexpr float kFloorFrom = -3e38f;
    static __device__ __forceinline__ uint32_t floor(float m)
    {
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rd(fmaxf(far_below(m), -3.38e38f)));
        return h | (h << 16);
    }
    static __device__ __forceinline__ float2 diff(const uint4 &v, int i, float2 nm, uint32_t fl)
    {
        uint32_t w;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w) : "r"((&v.x)[i]), "r"(fl));
        return add2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), nm);
    }
    // largest of a vector, NaN if it holds one
    static __device__ __forceinline__ float vmax(const uint4 &v)
    {
        uint32_t a, b;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a << 16)), "f"(__uint_as_float(a & 0xFFFF0000u)));
        return r;
    }
    static __device__ __forceinline__ float2 pair(const uint4 &v, int i)
    {
        const uint32_t w = (&v.x)[i];
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
};
template <>
struct LpType<__half> {
    static constexpr int VE = 8;
    static constexpr float kFloorFrom = -6e4f;
    static __device__ __forceinline__ uint32_t floor(float m)
    {
        const uint32_t h = __half_as_ushort(__float2half_rd(far_below(m)));
        return h | (h << 16);
    }
    static __device__ __forceinline__ float2 diff(const uint4 &v, int i, float2 nm, uint32_t fl)
    {
        uint32_t w;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(w) : "r"((&v.x)[i]), "r"(fl));
        return add2(__half22float2(*reinterpret_cast<const __half2 *>(&w)), nm);
    }
    static __device__ __forceinline__ float vmax(const uint4 &v)
    {
        uint32_t a, b;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(f.x), "f"(f.y));
        return r;
    }
    static __device__ __forceinline__ float2 pair(const uint4 &v, int i)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&(&v.x)[i]));
    }
};
template <>
struct LpType<float> {
    static constexpr int VE = 4;
    static constexpr float kFloorFrom = -INFINITY; // each difference is cut by itself
    static __device__ __forceinline__ uint32_t floor(float) { return 0; }
    static __device__ __forceinline__ float2 diff(const uint4 &v, int i, float2 nm, uint32_t)
    {
        return cut2(add2(pair(v, i), nm));
    }
    static __device__ __forceinline__ float vmax(const uint4 &v)
    {
        float a, b;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w)));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
        return a;
    }
    static __device__ __forceinline__ float2 pair(const uint4 &v, int i)
    {
        return make_float2(__uint_as_float((&v.x)[2 * i]), __uint_as_float((&v.x)[2 * i + 1]));
    }
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Bits that order like the value, -0 with +0 and every NaN above +inf.
__device__ __forceinline__ uint32_t order32(float f)
{
    uint32_t b = __float_as_uint(f);
    if (f != f)
        return 0xFFFFFFFFu;
    if (f == 0.f)
        b = 0;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float value32(uint32_t o)
{
    if (o == 0xFFFFFFFFu)
        return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// A candidate's key: order32, then the complement of its index.  Every key is
// above 0, which stands for "none" (the smallest order32, of -inf, is 0x007FFFFF).
constexpr uint32_t kOrderInf = 0xFF800000u; // order32(+inf)
constexpr uint32_t kOrderNan = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------
// Running softmax sums
// ---------------------------------------------------------------------------

__device__ __forceinline__ float diff_clamped(float x, float m) // NaN stays NaN
{
    float d = x - m;
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(kFarBelow));
    return d;
}

__device__ __forceinline__ float exp_2(float t)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}

__device__ __forceinline__ float exp_nat(float d)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * 1.4426950408889634f));
    return e;
}

struct Sums {
    float m, s, w; // maximum, sum of exp(x - m), sum of exp(x - m) (x - m)
};

__device__ __forceinline__ void rescale(Sums &a, float m)
{
    const float d = fmaxf(a.m - m, kFarBelow), c = exp_nat(d);
    a.w = c * fmaf(a.s, d, a.w);
    a.s *= c;
    a.m = m;
}

__device__ __forceinline__ void merge(Sums &a, Sums b)
{
    const float m = fmaxf(a.m, b.m);
    rescale(a, m);
    rescale(b, m);
    a.s += b.s;
    a.w += b.w;
}

// The sums of lanes 0 .. n-1 (a power of two, repeated over the warp) for every
// lane, each pair with the lower lane's first, so that all form the same sum.
__device__ __forceinline__ Sums butterfly(Sums t, int n)
{
    const int lane = threadIdx.x & 31;
    for (int o = n >> 1; o > 0; o >>= 1) {
        Sums x;
        x.m = __shfl_xor_sync(0xffffffffu, t.m, o);
        x.s = __shfl_xor_sync(0xffffffffu, t.s, o);
        x.w = __shfl_xor_sync(0xffffffffu, t.w, o);
        Sums lo = (lane & o) ? x : t, hi = (lane & o) ? t : x;
        merge(lo, hi);
        t = lo;
    }
    return t;
}

// ---------------------------------------------------------------------------
// Cluster (distributed shared memory)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float cluster_ld_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ key_t64 cluster_ld_u64(uint32_t a)
{
    key_t64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------

// A value that at least k of the threads' keys reach, and at most lp_accept(k)
// of them unless too many are equal to the k-th largest; 0 if fewer than k
// threads have a key.  top: no key is above it.  reach: the threads that reach it.
// Called by the whole CTA.
__device__ __forceinline__ uint32_t bound_of_threads(uint32_t mine, uint32_t top, int k, int &reach)
{
    reach = __syncthreads_count(mine != 0);
    if (reach < k)
        return 0;
    // from the top down in growing steps (the maxima of many logits lie close
    // together), then by halves
    uint32_t lo = 0, hi = top; // at least k reach lo; fewer than k reach anything above hi
    uint32_t step = 1u << 20;
    while (lo < hi) {
        uint32_t mid = hi - (hi - lo) / 2; // above lo
        if (lo == 0 && step < hi - mid)
            mid = hi - step;
        const int c = __syncthreads_count(mine >= mid);
        if (c >= k)
            reach = c;
        if (c >= k && c <= lp_accept(k))
            return mid;
        if (c < k) {
            hi = mid - 1;
            if (step < (1u << 30))
                step <<= 1;
        } else {
            lo = mid;
        }
    }
    return lo;
}

// The sum of c over the CTA, for everyone; slot alternates between calls.
__device__ __forceinline__ int block_sum(int c, int *s_count, int &slot)
{
    if (threadIdx.x == 0)
        s_count[slot] = 0;
    __syncthreads();
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0 && c)
        atomicAdd(&s_count[slot], c);
    __syncthreads();
    c = s_count[slot];
    slot ^= 1; // the word just read is written again after the next call's barriers
    return c;
}

// A bound that between k and lp_accept(k) of the n >= k different keys of a list
// reach.
__device__ __forceinline__ key_t64 bound_of_list(const key_t64 *list, int n, int k, int *s_count)
{
    key_t64 lo = 0, hi = ~0ull; // at least k reach lo; fewer than k (or the accepted few) reach hi
    for (int slot = 0;;) {
        const key_t64 mid = lo + (hi - lo) / 2;
        if (mid == lo)
            return lo;
        int c = 0;
        for (int i = threadIdx.x; i < n; i += blockDim.x)
            c += list[i] >= mid;
        c = block_sum(c, s_count, slot);
        if (c >= k && c <= lp_accept(k))
            return mid;
        if (c < k)
            hi = mid;
        else
            lo = mid;
    }
}

// Ranks the n keys of src (n <= kSortMax, all different) by counting, the k
// largest in order into dst, 0 behind them if there are fewer.
__device__ __forceinline__ void rank_into(const key_t64 *src, int n, int k, key_t64 *dst)
{
    for (int i = threadIdx.x; i < k; i += blockDim.x)
        if (i >= n)
            dst[i] = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const key_t64 mine = src[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            above += src[j] > mine;
        if (above < k)
            dst[above] = mine;
    }
    __syncthreads();
}

struct LpShared {
    key_t64 list[kListMax];  // candidates
    key_t64 cut[kSortMax];   // a list cut back before it is ranked
    key_t64 best[kTopkMaxK]; // this CTA's k best, in order
    key_t64 others[kLpMaxCluster * kTopkMaxK];
    Sums warp_sums[32];
    Sums sums; // this CTA's
    // runs of vectors that may hold one of the k largest: the thread that read
    // them, and the run's number among its own in the upper half
    uint32_t chosen[kChosenMax];
    int chosen_count, count, cut_count, list_count[2];
    int place[kTopkMaxK];
    int warp_count[32];
};

// The list's k best, in order, into sh.best.
template <class Shared>
__device__ __forceinline__ void sort_list(Shared &sh, int n, int k)
{
    if (n <= kSortMax) {
        rank_into(sh.list, n, k, sh.best);
        return;
    }
    const key_t64 b = bound_of_list(sh.list, n, k, sh.list_count);
    if (threadIdx.x == 0)
        sh.cut_count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (sh.list[i] >= b)
            sh.cut[atomicAdd(&sh.cut_count, 1)] = sh.list[i]; // at most lp_accept(k) <= kSortMax
    __syncthreads();
    rank_into(sh.cut, sh.cut_count, k, sh.best);
}

// A CTA's slice of a row: elements [e0, e1), of which [v0, v0 + nv VE) are whole
// aligned vectors, vector i read by thread i mod THREADS, and the up to 2 VE - 2
// others, before and behind them, by one thread each.
template <class T, int THREADS>
struct Slice {
    static constexpr int VE = LpType<T>::VE;
    const T *row;
    int e0, e1, v0, nv;
    __device__ __forceinline__ Slice(const T *row_, int e0_, int e1_) : row(row_), e0(e0_), e1(e1_)
    {
        const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(row + e0) & 15)) & 15) / (int)sizeof(T);
        v0 = min(e1, e0 + lead);
        nv = (e1 - v0) / VE;
    }
    __device__ __forceinline__ const uint4 *vec() const { return reinterpret_cast<const uint4 *>(row + v0); }
    __device__ __forceinline__ int edge() const // this thread's element outside the vectors, or -1
    {
        const int t = threadIdx.x, n0 = v0 - e0, tail = v0 + nv * VE;
        return t < n0 ? e0 + t : t < n0 + e1 - tail ? tail + t - n0 : -1;
    }
};

// Elements of the chosen runs of `per` vectors and of the edges whose order32 is
// above o (at least o with or_equal): f(order32, index) for each, from any
// thread.
template <class T, int THREADS, class Shared, class F>
__device__ __forceinline__ void each_above(const Slice<T, THREADS> &sl, const Shared &sh, int per, uint32_t o,
                                           bool or_equal, F f)
{
    using L = LpType<T>;
    constexpr int VE = L::VE;
    const int items = sh.chosen_count * per;
    const float inv = 1.f / (float)per;
    const float of = value32(o); // a NaN passes, and lets everything pass
    constexpr int G = 4;         // vectors in flight
    for (int i0 = threadIdx.x; i0 < items; i0 += G * THREADS) {
        uint4 q[G];
        int v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // i / per: i < 2^18, so (i + 1/2) / per is off by less than its distance
            // to a whole number, 1 / (2 per)
            const int i = i0 + g * THREADS, c = (int)(((float)i + 0.5f) * inv);
            v[g] = sl.nv;
            if (i < items) {
                const uint32_t run = sh.chosen[c];
                v[g] = ((int)(run >> 16) * per + i - c * per) * THREADS + (int)(run & 0xFFFFu);
            }
            if (v[g] < sl.nv)
                q[g] = __ldg(sl.vec() + v[g]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (v[g] >= sl.nv || L::vmax(q[g]) < of)
                continue;
#pragma unroll
            for (int j = 0; j < VE / 2; ++j) {
                const float2 x = L::pair(q[g], j);
                const uint32_t a = order32(x.x), b = order32(x.y);
                if (a > o || (or_equal && a == o))
                    f(a, sl.v0 + v[g] * VE + 2 * j);
                if (b > o || (or_equal && b == o))
                    f(b, sl.v0 + v[g] * VE + 2 * j + 1);
            }
        }
    }
    const int e = sl.edge();
    if (e >= 0) {
        const uint32_t a = order32(to_float(sl.row[e]));
        if (a > o || (or_equal && a == o))
            f(a, e);
    }
}

// Appends the first `want` elements equal to order32 o of the slice, in index
// order, behind the `have` entries of the list.
template <class T, int THREADS, class Shared>
__device__ __noinline__ void first_equal(const Slice<T, THREADS> &sl, Shared &sh, uint32_t o, int have, int want)
{
    using L = LpType<T>;
    constexpr int VE = L::VE;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = sl.v0 - sl.e0, tail = sl.v0 + sl.nv * VE;
    // rounds of up to VE consecutive elements a thread: the lead, THREADS vectors at a time, the tail
    const int rounds = 2 + (sl.nv + THREADS - 1) / THREADS;
    for (int r = 0; r < rounds && want > 0; ++r) {
        uint32_t hit = 0; // bit j: element j of this thread's run equals o
        int at = 0;
        if (r == 0 || r == rounds - 1) {
            at = r == 0 ? sl.e0 + (int)threadIdx.x : tail + (int)threadIdx.x;
            if ((int)threadIdx.x < (r == 0 ? n0 : sl.e1 - tail))
                hit = order32(to_float(sl.row[at])) == o;
        } else {
            const int v = (r - 1) * THREADS + (int)threadIdx.x;
            at = sl.v0 + v * VE;
            if (v < sl.nv) {
                const uint4 q = __ldg(sl.vec() + v);
#pragma unroll
                for (int j = 0; j < VE / 2; ++j) {
                    const float2 x = L::pair(q, j);
                    hit |= (uint32_t)(order32(x.x) == o) << (2 * j) | (uint32_t)(order32(x.y) == o) << (2 * j + 1);
                }
            }
        }
        const int c = __popc(hit);
        int inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d)
                inc += u;
        }
        if (lane == 31)
            sh.warp_count[warp] = inc;
        __syncthreads();
        int before = inc - c, total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            before += w < warp ? sh.warp_count[w] : 0;
            total += sh.warp_count[w];
        }
        for (int j = 0; hit; ++j, hit >>= 1)
            if ((hit & 1u) && before < want) {
                sh.list[have + before] = ((key_t64)o << 32) | (uint32_t)~(at + j);
                ++before;
            }
        __syncthreads(); // warp_count is written again
        have += min(total, want);
        want -= min(total, want);
    }
}

// For a slice with many logits equal to `bound` (a mask that leaves few others),
// which at least k logits reach: lists those above it, from the runs that hold one,
// and the first of the equal ones behind them.  Returns the list's length, at
// least k, or 0 if there are too many above it, too.
template <class T, int THREADS, class Shared>
__device__ __noinline__ int list_above(const Slice<T, THREADS> &sl, Shared &sh, uint32_t bound, int k,
                                       const float *runs, int per_run, int n_runs)
{
    __syncthreads(); // every thread has read sh.chosen_count
    if (threadIdx.x == 0)
        sh.chosen_count = 0;
    __syncthreads();
    const float of = value32(bound);
    for (int i = 0; i < n_runs; ++i)
        if (runs[i * THREADS] > of) {
            const int at = atomicAdd(&sh.chosen_count, 1);
            if (at < kChosenMax)
                sh.chosen[at] = (uint32_t)i << 16 | threadIdx.x;
        }
    __syncthreads();
    if (sh.chosen_count > kChosenMax)
        return 0;
    each_above(sl, sh, per_run, bound, false, [&](uint32_t o, int idx) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kListMax)
            sh.list[at] = ((key_t64)o << 32) | (uint32_t)~idx;
    });
    __syncthreads();
    const int n = sh.count;
    if (n > kListMax) {
        __syncthreads();
        if (threadIdx.x == 0)
            sh.count = 0; // the caller's
        return 0;
    }
    if (n >= k)
        return n;
    first_equal(sl, sh, bound, n, k - n);
    __syncthreads();
    return k;
}

// The slice's k best, in order, into sh.best.  mine: order32 that the largest
// logit this thread read reaches, 0 if it read none; top: no logit is above it;
// runs: the largest of each run of per_run vectors this thread read, THREADS
// apart (nan: one may be hidden in them).
template <class T, int THREADS, class Shared>
__device__ __forceinline__ void select_best(const Slice<T, THREADS> &sl, Shared &sh, uint32_t mine, uint32_t top, int k,
                                            const float *runs, int per_run, bool nan)
{
    if (threadIdx.x == 0)
        sh.chosen_count = sh.count = 0;
    int reach;
    const uint32_t bound = bound_of_threads(mine, min(top, kOrderInf), k, reach); // has a barrier
    const int all = (sl.nv + THREADS - 1) / THREADS; // vectors of a thread, at most
    const bool chosen = mine != 0 && mine >= bound;
    if (chosen) {
        const float of = value32(bound);
        const int n = (all + per_run - 1) / per_run;
        for (int i0 = 0; i0 < n; i0 += 8) {
            uint32_t hit = 0; // eight at a time: the loads overlap
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < n)
                    hit |= (uint32_t)(nan || !(runs[(i0 + i) * THREADS] < of)) << i;
            if (hit == 0)
                continue;
            int at = atomicAdd(&sh.chosen_count, __popc(hit));
            for (; hit; hit &= hit - 1, ++at)
                if (at < kChosenMax)
                    sh.chosen[at] = (uint32_t)(i0 + __ffs(hit) - 1) << 16 | threadIdx.x;
        }
    }
    __syncthreads();
    int per = per_run;
    bool columns = sh.chosen_count > kChosenMax;
    // Many threads reach the bound and none could be told from another: a value that
    // much of the row shares.  (16-bit logits at large have ties, too, but not of three
    // threads in four.)
    if (top != kOrderNan && (columns || (bound != 0 && reach > lp_accept(k) && reach > THREADS * 3 / 4))) {
        const int n = list_above(sl, sh, bound, k, runs, per_run, (all + per_run - 1) / per_run);
        if (n) {
            sort_list(sh, n, k);
            return;
        }
        columns = true;
    }
    if (columns) {
        // too many runs: the chosen threads' whole columns
        per = all;
        __syncthreads();
        if (threadIdx.x == 0)
            sh.chosen_count = 0;
        __syncthreads();
        if (chosen)
            sh.chosen[atomicAdd(&sh.chosen_count, 1)] = threadIdx.x;
        __syncthreads();
    }
    each_above(sl, sh, per, bound, true, [&](uint32_t o, int idx) {
        if (*(volatile int *)&sh.count > kListMax)
            return; // too many already: a masked row's thousands would queue for the counter
        const int at = atomicAdd(&sh.count, 1);
        if (at < kListMax)
            sh.list[at] = ((key_t64)o << 32) | (uint32_t)~idx;
    });
    __syncthreads();
    int n = sh.count;
    if (n > kListMax) {
        // the k-th largest value: the largest that at least k elements reach
        uint32_t lo = bound, hi = top;
        int slot = 0;
        while (lo < hi) {
            const uint32_t mid = hi - (hi - lo) / 2;
            int c = 0;
            each_above(sl, sh, per, mid, true, [&](uint32_t, int) { ++c; });
            if (block_sum(c, sh.list_count, slot) >= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        __syncthreads(); // every thread has read sh.count
        if (threadIdx.x == 0)
            sh.count = 0;
        __syncthreads();
        each_above(sl, sh, per, lo, false, [&](uint32_t o, int idx) { // fewer than k
            sh.list[atomicAdd(&sh.count, 1)] = ((key_t64)o << 32) | (uint32_t)~idx;
        });
        __syncthreads();
        n = sh.count;
        first_equal(sl, sh, lo, n, k - n);
        __syncthreads();
        n = k;
    }
    sort_list(sh, n, k);
}

template <class T, int THREADS, bool TOPK>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const LpParams p)
{
    using L = LpType<T>;
    constexpr int VE = L::VE, B = THREADS * kUnroll; // vectors per batch
    __shared__ LpShared sh;
    extern __shared__ float s_runs[]; // [kRuns][THREADS] (TOPK)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = p.C > 1 ? (int)cluster_rank() : 0;
    const int m = blockIdx.x / p.C, k = p.k;

    pdl_launch_dependents();
    pdl_wait(); // the logits may come from the preceding kernel

    const T *row = static_cast<const T *>(p.logits) + (long long)m * p.ld;
    const int e0 = min(p.N, rank * p.slice);
    const Slice<T, THREADS> sl(row, e0, min(p.N, e0 + p.slice));
    const int nv = sl.nv;
    const uint4 *vec = sl.vec();

    int token = -1;
    float x_token = 0.f;
    if (rank == 0 && threadIdx.x == 0 && p.tokens) {
        token = p.tokens[m];
        if (token >= 0 && token < p.N)
            x_token = to_float(row[token]);
    }

    constexpr uint32_t minus_inf = std::is_same_v<T, float> ? 0xFF800000u
                                   : std::is_same_v<T, __half> ? 0xFC00FC00u
                                                               : 0xFF80FF80u;
    const uint4 none = make_uint4(minus_inf, minus_inf, minus_inf, minus_inf);
    uint4 cur[kUnroll], nxt[kUnroll];
    auto load = [&](int b, uint4(&v)[kUnroll]) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = b + u * THREADS + (int)threadIdx.x;
            v[u] = i < nv ? ldg_stream(vec + i) : none;
        }
    };
    load(0, cur);

    Sums a{-FLT_MAX, 0.f, 0.f};
    float largest = -INFINITY; // a.m starts at the lowest finite value, above -inf
    const int edge = sl.edge();
    if (edge >= 0) {
        const float x = to_float(row[edge]);
        largest = x;
        a.m = fmaxf(a.m, x);
        const float d = diff_clamped(x, a.m);
        a.s = exp_nat(d);
        a.w = a.s * d;
    }

    int run = 0, in_run = 0; // of this batch
    float run_max = -INFINITY;
    for (int b = 0; b < nv; b += B) {
        if (b + B < nv)
            load(b + B, nxt);
        float bm = L::vmax(cur[0]); // fmaxf below drops a NaN; the sums keep it
#pragma unroll
        for (int u = 1; u < kUnroll; ++u)
            bm = fmaxf(bm, L::vmax(cur[u]));
        largest = fmaxf(largest, bm);
        if constexpr (TOPK) {
            run_max = fmaxf(run_max, bm);
            s_runs[run * THREADS + threadIdx.x] = run_max;
            if (++in_run == p.run_batches) {
                ++run;
                in_run = 0;
                run_max = -INFINITY;
            }
        }
        if (bm > a.m)
            rescale(a, bm);
        float2 s2 = make_float2(0.f, 0.f), w2 = s2;
        const float2 nm = make_float2(-a.m, -a.m);
        const uint32_t fl = L::floor(a.m);
        auto add = [&](bool fast) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                const float2 d = fast ? L::diff(cur[u], i, nm, fl) : cut2(add2(L::pair(cur[u], i), nm));
                const float2 t = mul2(d, make_float2(1.4426950408889634f, 1.4426950408889634f));
                const float2 e = make_float2(exp_2(t.x), exp_2(t.y));
                s2 = add2(s2, e);
                w2 = fma2(e, d, w2);
            }
        };
        if (a.m >= L::kFloorFrom)
            add(true);
        else
            add(false);
        a.s += s2.x + s2.y;
        a.w += w2.x + w2.y;

#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            cur[u] = nxt[u];
    }

    // order32 of this thread's largest, or, where a NaN sum tells of a NaN or +inf
    // in it, what it reaches at least
    const bool a_nan = a.s != a.s;
    uint32_t mine = 0;
    if (edge >= 0 || (int)threadIdx.x < nv)
        mine = a_nan ? kOrderInf : order32(largest);

    // ---- the CTA's sums: lanes, then warps, in a fixed order ----
    {
        float mx = a.m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        rescale(a, mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) { // both sides of an exchange form the same sum
            a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
            a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
        }
    }
    if (lane == 0)
        sh.warp_sums[warp] = a;
    __syncthreads(); // also: s_runs is written
    constexpr int W = THREADS / 32;
    Sums t = sh.warp_sums[lane & (W - 1)]; // every warp, the same sums in the same order
    t = butterfly(t, W);
    if constexpr (TOPK)
        select_best(sl, sh, mine, t.s != t.s ? kOrderNan : order32(t.m), k, s_runs + threadIdx.x,
                    p.run_batches * kUnroll, a_nan);
    if (p.C > 1) {
        if (threadIdx.x == 0)
            sh.sums = t;
        cluster_sync();
        { // lane c holds CTA c's sums (p.C is a power of two)
            const uint32_t at = cluster_addr(&sh.sums, lane & (p.C - 1));
            t.m = cluster_ld_f32(at);
            t.s = cluster_ld_f32(at + 4);
            t.w = cluster_ld_f32(at + 8);
        }
        if constexpr (TOPK)
            for (int i = threadIdx.x; i < p.C * k; i += THREADS)
                sh.others[i] = cluster_ld_u64(cluster_addr(&sh.best[i % k], i / k));
        t = butterfly(t, p.C);
        cluster_sync(); // no CTA leaves while another reads its shared memory
    }
    const float log_s = logf(t.s);
    if (rank == 0 && threadIdx.x == 0) {
        if (p.logprob)
            p.logprob[m] = token >= 0 && token < p.N ? (x_token - t.m) - log_s : __uint_as_float(0x7FFFFFFFu);
        if (p.entropy)
            p.entropy[m] = log_s - t.w / t.s;
    }
    if constexpr (TOPK) {
        // an entry's place: its own list's, and the entries above it in the others
        if (p.C > 1) {
            for (int i = threadIdx.x; i < k; i += THREADS)
                sh.place[i] = i;
            __syncthreads();
            for (int i = threadIdx.x; i < p.C * k; i += THREADS) {
                const int c = i / k, e = i - c * k;
                if (c == rank)
                    continue;
                const key_t64 key = sh.best[e], *o = sh.others + c * k;
                int lo = 0, hi = k; // entries of a descending list above key
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (o[mid] > key)
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                if (lo)
                    atomicAdd(&sh.place[e], lo);
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < k; i += THREADS) {
            const key_t64 key = sh.best[i];
            const int at = p.C > 1 ? sh.place[i] : i;
            if (key != 0 && at < k) { // 0: this slice is shorter than k
                p.top[(size_t)m * k + at] = (value32((uint32_t)(key >> 32)) - t.m) - log_s;
                p.top_idx[(size_t)m * k + at] = (int32_t)~(uint32_t)key;
            }
        }
    }
}

template <class T, int THREADS, bool TOPK>
cudaError_t launch_lp(LpParams p, int sm_count, cudaStream_t st)
{
    constexpr int VE = LpType<T>::VE;
    // CTAs of a row: while they fit the GPU at once with the others', and each
    // has a batch's work at least
    const long long slots = (long long)sm_count * (1024 / THREADS);
    int C = 1;
    while (C < kLpMaxCluster && (long long)p.M * C * 2 <= slots && p.N / (2 * C) >= THREADS * VE)
        C *= 2;
    p.C = C;
    p.slice = ((p.N + C - 1) / C + VE - 1) / VE * VE;
    const int batches = (p.slice + THREADS * kUnroll * VE - 1) / (THREADS * kUnroll * VE);
    p.run_batches = (batches + kRuns - 1) / kRuns;
    const int runs = p.run_batches ? (batches + p.run_batches - 1) / p.run_batches : 0;
    const size_t smem = TOPK ? (size_t)runs * THREADS * sizeof(float) : 0;
    const cudaError_t e = kernel_setup((const void *)logprobs_kernel<T, THREADS, TOPK>, smem, 0, 0, nullptr);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    cfg.gridDim = dim3((unsigned)p.M * C);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, THREADS, TOPK>, p);
}

template <class T, int THREADS>
cudaError_t launch_lp_size(const LpParams &p, int sm_count, cudaStream_t st)
{
    return p.k > 0 ? launch_lp<T, THREADS, true>(p, sm_count, st) : launch_lp<T, THREADS, false>(p, sm_count, st);
}

template <class T>
cudaError_t launch_lp_type(const LpParams &p, int sm_count, cudaStream_t st)
{
    // Short rows on small CTAs, eight to an SM: what a CTA does besides reading
    // (barriers, the search, the ranking) is then spread over more rows.
    const bool small = p.N <= kShortBatches * 128 * kUnroll * LpType<T>::VE;
    return small ? launch_lp_size<T, 128>(p, sm_count, st) : launch_lp_size<T, 256>(p, sm_count, st);
}

} // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int M, int N, long long ld, const int32_t *tokens, int k,
                            float *logprob, float *entropy, float *top, int32_t *top_idx, int sm_count,
                            cudaStream_t st)
{
    LpParams p{logits, ld, M, N, k, 1, N, 1, tokens, logprob, entropy, top, top_idx};
    switch (dtype) {
    case WQ_DTYPE_BF16: return launch_lp_type<__nv_bfloat16>(p, sm_count, st);
    case WQ_DTYPE_F16: return launch_lp_type<__half>(p, sm_count, st);
    default: return launch_lp_type<float>(p, sm_count, st);
    }
}

} // namespace wq
