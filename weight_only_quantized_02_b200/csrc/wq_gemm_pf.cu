// wq_gemm_pf.cu -- the layer over a prompt: W8A16 and W4A16 (group 128) for
// many tokens, on pairs of SMs.
//
//     v[m][n] = s[n] sum_k q[n][k] x[m][k]                        (INT8)
//     v[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[m][k]   (INT4)
//
// then the epilogue (wq_epilogue.cuh).  The tensor cores take the exact
// integers q and q - z in the activations' format; the only rounding before
// the epilogue is the fp32 accumulation.
//
// Bound: the tensor cores.  Two CTAs (a cluster, one on each SM of a pair)
// work on one tile of 256 output channels with tcgen05.mma.cta_group::2: each
// CTA holds its own 128 channels' weights and accumulators in its tensor memory
// and half of the tokens' activations in its shared memory, so an activation
// byte is brought in once for 256 channels.  A CTA alone (128 channels) would
// have to fill twice that, more than L2 gives an SM in the time of its products.
//
// Tensor memory: two accumulators of 192 columns (tokens) and two A stages of
// 64 columns (128 k of dequantized weights).
//   INT4: a tile is one accumulator's 192 tokens; a group's sums are retired
//         into fp32 register totals while the next group is multiplied into the
//         other accumulator.
//   INT8: a tile is both accumulators, 384 tokens, so that a dequantized block
//         is multiplied twice: at 192 tokens the dequantization, some 600
//         cycles a 64-k step against 384 of products, held the tensor cores back.
// M is cut into equal tiles, rounded up to 16 tokens, so ragged prompts waste
// little.
//
// Work: units (tile, 128-k block), tiles of one channel panel pair next to each
// other; each pair of CTAs takes an equal contiguous run of units (stream-K,
// the partial sums of a tile that two or more pairs share are added in their
// order by the last to arrive), or whole tiles where there is no workspace.
//
// Warps (20; registers are moved to the roles that need them):
//   0      x producer: the CTA's half of the tile's tokens, 64 k a stage (tensor
//          map, 128-byte swizzle), signalled on the leader's barrier
//   1      weight producer: a unit's packed block (and zero points)
//   2      tensor memory; in the leader CTA, the lane that issues the MMAs
//   4-11   retire warps: lane quadrant x half of the token columns; INT4 scales go
//          from global memory to a register two groups ahead (through shared
//          memory and a barrier of their own they took 280 cycles a group)
//   12-19  dequantization: packed block -> exact integers in tensor memory
// One commit for each 64 k, to both CTAs, tells the x producers (8 or 4 stages),
// the dequantization (2 units) and, for INT4, the retire warps (2 groups) that
// the products are done.
//
// Measured on B200 (layer with a residual or the other half of a gate, the weights
// in L2): INT4 17408 x 5120, 2048 tokens 360 us (1014 TFLOP/s); 5120 x 17408, 364
// tokens 82; INT8 17408 x 5120, 2048 tokens 314 (1170 TFLOP/s); 5120 x 17408, 333
// tokens 58.  In one launch of 2048 tokens the tensor pipe is busy in 70 % of the
// cycles for INT8, at 1.57 GHz (back to back, the power limit holds the clock
// between 1.0 and 1.4 and the pipe is nearly always busy), and in 51 % for INT4, at
// 1.66 GHz.  INT4 is held by the work beside the products: a unit takes some 1350
// cycles against 768 of products at 192 tokens, the dequantization about 1200 of its
// warps' time and the retirement 900, both by instruction latency at one or two
// warps a scheduler; neither alone (a third of the retirement 320 us, no conversion
// of the codes 327).
//
// Every wait is bounded (2 s); a timeout is recorded, every role winds down, and a
// producer waits (as long at most) for its copies in flight before the CTAs leave.
#include <atomic>
#include <cstdint>

#include "wq.h"
#include "wq_device.cuh"
#include "wq_epilogue.cuh"
#include "wq_gemm_common.cuh"
#include "wq_internal.h"

namespace wq {

static __device__ int g_gemm_pf_error = 0;

namespace {

constexpr int kPfTok = 192;       // columns of an accumulator
constexpr int kPfA0 = 2 * kPfTok; // first A column
constexpr int kPfXB = kPfTok / 2 * 128;       // bytes of 64 k of an accumulator's tokens, one CTA's half
constexpr int kPfOutB = 16 * kPanelRows * 4;  // 16 tokens of a CTA's channels on their way out, fp32
static_assert(kPfA0 + 2 * 64 == 512, "tensor memory plan");

template <int BITS>
struct PfCfg {
    static constexpr int kWB = BITS == 4 ? 8192 : 16384;
    static constexpr int kWS = BITS == 4 ? 8 : 4;   // weight stages (units)
    static constexpr int kSub = BITS == 4 ? 1 : 2;  // accumulators of a tile
    static constexpr int kXS = 8 / kSub;            // x stages (64 k)
    static constexpr int kUnroll = kXS / 2;         // units of one round of the x ring
    static constexpr int kXB = kSub * kPfXB;
    static constexpr int kAH = kSub;          // 64-k halves of an A stage (32 columns each)
    static constexpr int kAS = 4 / kAH;       // A stages
    // retire warps: groups of four (one a lane quadrant) that share an
    // accumulator's columns
    static constexpr int kGroups = 2;
    static constexpr int kChunks = kPfTok / 16 / kGroups; // 16-column chunks of one, at most
    static constexpr int kThreads = 128 + kGroups * 128 + 256;
    // registers a thread at launch, and by role
    static constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
    static constexpr int kRegsIssue = 32, kRegsRetire = BITS == 4 ? 176 : 144,
                         kRegsDequant = BITS == 4 ? 48 : 80;
    static constexpr int kRegs = 128 * kRegsIssue + kGroups * 128 * kRegsRetire + 256 * kRegsDequant;
    static_assert(kRegs <= kThreads * kRegsLaunch, "the roles' registers come out of the CTA's at launch");
    static_assert(kUnroll % 2 == 0, "a unit's A stage and accumulator are constants of the unrolled loops");
};

struct PfParams {
    int M, N, KB, U, TT, n, nsub, tiles, panels; // n: tokens of an accumulator (a multiple of 16); nsub of them a tile
    int align;                             // 1: whole tiles per pair
    const uint8_t *wq;
    const uint16_t *scales;
    const uint8_t *zeros;
    uint16_t *y;
    EpiArgs epi;
    float *part;   // [pairs][2 slots][2 CTAs][nsub n tokens][128 rows]
    uint32_t *cnt; // [pairs][2 CTAs][kGroups], by a split tile's first pair
};

template <int BITS>
constexpr size_t pf_smem_bytes()
{
    using C = PfCfg<BITS>;
    return 1024 + (size_t)C::kXS * C::kXB + (size_t)C::kWS * C::kWB + 2 * C::kGroups * kPfOutB +
           (size_t)C::kWS * 128 + (size_t)(2 * C::kXS + 2 * C::kWS + C::kAS + 4) * 8 + 32;
}

// ---- pairs of CTAs ----
__device__ __forceinline__ uint32_t pf_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t pf_map(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// Arrival on a barrier of either CTA.  What it hands over is in tensor memory,
// ordered by tcgen05.fence; a release at cluster scope, which it does not need,
// took 1400 cycles.
// One lane's (who) arrival for its warp, by predicate: the tensor-memory
// instructions around it are the whole warp's, and a branch could leave the warp
// split on the way to the next of them.  (Where code branches by lane on that way,
// a __syncwarp or a vote stands before the next one.)
__device__ __forceinline__ void pf_arrive(uint32_t cluster_bar, bool who)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_bar),
                 "r"((uint32_t)who)
                 : "memory");
}
__device__ __forceinline__ void pf_arrive_own(uint64_t *bar, bool who) // a barrier of this CTA
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
                 "r"((uint32_t)who)
                 : "memory");
}
// Barrier of the four warps of a retire group, and whether all of them are well.
__device__ __forceinline__ bool pf_all(int id, bool ok)
{
    uint32_t r;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
                 "barrier.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(128), "r"((uint32_t)ok)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ bool pf_elect() // one lane of the (converged) warp
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void pf_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void pf_tmem_alloc(uint32_t *dst)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pf_tmem_dealloc(uint32_t taddr)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
// x box into this CTA's shared memory, completing on the leader's barrier.
__device__ __forceinline__ void pf_load_x(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t cluster_bar,
                                          uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(c0), "r"(c1), "r"(cluster_bar), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void pf_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// Arrives on the barrier at this address in both CTAs when the MMAs issued so
// far have completed.
__device__ __forceinline__ void pf_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// d += {a, a} {b0, b1}, a pair of fp32 sums kept packed (each half rounded as fmaf).
__device__ __forceinline__ void pf_ffma2(unsigned long long &d, unsigned long long aa, float b0, float b1)
{
    unsigned long long bb;
    asm("mov.b64 %0, {%1, %2};" : "=l"(bb) : "f"(b0), "f"(b1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(aa), "l"(bb));
}

// Exact integers in the activations' format.
template <bool F16>
__device__ __forceinline__ uint32_t pf_sub2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (F16)
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two int8 codes (bytes 2 h, 2 h + 1 of w).  bf16: with the low seven bits,
// 0x4300 | c is 128 + c; with the sign bit, 0x4300 | 0x80 is 256.  fp16: 0x6400 | c
// is 1024 + c for the code plus 128 (its sign bit turned over).
template <bool F16>
__device__ __forceinline__ uint32_t pf_s8pair(uint32_t w, int h)
{
    if constexpr (F16)
        return pf_sub2<true>(__byte_perm(w ^ 0x80808080u, 0x64646464u, h == 0 ? 0x4140u : 0x4342u), 0x64806480u);
    const uint32_t b = __byte_perm(w, 0u, h == 0 ? 0x4140u : 0x4342u);
    uint32_t mag, off;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(mag) : "r"(b), "r"(0x007F007Fu), "r"(0x43004300u));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(off) : "r"(b), "r"(0x00800080u), "r"(0x43004300u));
    return pf_sub2<false>(mag, off);
}

// One INT4 tile (16 rows x 64 k) as int4_tile_regs has it, in either format:
// zlo, zhi are the format's {magic + z} pairs of this lane's two rows.
template <bool F16>
constexpr uint32_t kPfMagic2 = F16 ? 0x64006400u : 0x43004300u;
template <bool F16>
__device__ __forceinline__ void pf_int4_regs(const uint4 &w, uint32_t zlo, uint32_t zhi, uint32_t (&r)[16])
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) // words x, y, z, w: rows lo, hi, lo, hi; registers 8 (i / 2) + 2 (i % 2) + ...
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t n;
            asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(n) : "r"(v[i] >> (4 * j)), "r"(0x000F000Fu), "r"(kPfMagic2<F16>));
            r[8 * (i / 2) + 2 * (i % 2) + 4 * (j / 2) + j % 2] = pf_sub2<F16>(n, i % 2 ? zhi : zlo);
        }
}

// First unit of pair c.
__device__ __forceinline__ int pf_start(const PfParams &p, int G, int c)
{
    return p.align ? sk_start(p.tiles, G, c) * p.KB : sk_start(p.U, G, c);
}

// The pair whose range holds unit u: the last one that starts at or before it.
__device__ __forceinline__ int pf_owner(const PfParams &p, int G, int u)
{
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pf_start(p, G, mid) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Waits (bounded) until the last of n copies into a ring of `stages` have landed: a
// producer whose wait gave up does not leave them in flight behind its CTA.  (Of a
// producer that came to its end the MMA issuer waits for every copy, or gives up
// after longer than any takes.)
__device__ __noinline__ void pf_landed(uint64_t *full, int stages, int n)
{
    for (int j = max(0, n - stages); j < n; ++j)
        if (!mbar_wait(&full[j % stages], (j / stages) & 1))
            return;
}

// What a retire warp needs to write a tile out.
struct PfRetire {
    int ch0, nc; // the warp's group: first 16-token chunk of an accumulator, chunks
    int G, pair, rank, u0, u1;
    float *obuf;      // the group's two output buffers
    uint32_t *ticket; // the group's shared word
    uint32_t ebar;    // the leader's accempty barriers
    uint32_t tq;      // the warp's corner of accumulator 0
};

// The output path: 16 tokens (a chunk) of the CTA's 128 channels at a time.  The
// group's four warps put their sums into shared memory, a channel a thread, and
// take them out as 8 consecutive channels of a token a thread, so that y and
// the operands move in 16-byte pieces, 256 contiguous bytes a token.  (Written
// 2 bytes a lane, 64 a warp, a tile with a residual took 38 us to leave.)
template <bool F16>
struct PfOut {
    // copies: the launch parameters are behind a pointer here, and would be read
    // again after every barrier
    const int M, N, n, nc, act, out_f32;
    const int tok0;         // this thread's first token of the tile, less 16 times the chunk
    const int step1;        // from the first accumulator's last chunk to the second's first, less 16
    const long long ld_mul, ld_res;
    uint16_t *const y;
    const uint16_t *const pmul, *const pres;
    float *const obuf;
    const int r, og, ot, id, nn; // channel written to shared memory; channels nn .. nn + 7 (og of the CTA's) and token taken out
    int ob;
    bool vec_mul, vec_res;
    uint4 mul[2], res[2]; // the operands of this thread's two tokens of the next chunk
    float bias[8];

    // r: the retire warps start at warp 4, so a thread's place in its group is its
    // lane quadrant's row
    __device__ __forceinline__ PfOut(const PfParams &p, const PfRetire &rt, int tile)
        : M(p.M), N(p.N), n(p.n), nc(rt.nc), act(p.epi.act), out_f32(p.epi.out_f32),
          tok0((tile % p.TT) * p.nsub * p.n + 16 * rt.ch0 + ((int)(threadIdx.x & 127) >> 4)),
          step1(p.n - 16 * rt.nc), ld_mul(p.epi.ld_mul), ld_res(p.epi.ld_res), y(p.y), pmul(p.epi.mul),
          pres(p.epi.res), obuf(rt.obuf), r(threadIdx.x & 127), og(8 * (threadIdx.x & 15)),
          ot((threadIdx.x & 127) >> 4), id(1 + ((threadIdx.x - 128) >> 7)),
          nn((2 * (tile / p.TT) + rt.rank) * kPanelRows + 8 * (int)(threadIdx.x & 15))
    {
        ob = 0; // the group has met since the buffers were last read
        vec_mul = ((reinterpret_cast<uintptr_t>(pmul) | (uintptr_t)(2 * ld_mul)) & 15) == 0;
        vec_res = ((reinterpret_cast<uintptr_t>(pres) | (uintptr_t)(2 * ld_res)) & 15) == 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            bias[j] = p.epi.bias && nn < N ? act16_to_float<F16>(__ldg(p.epi.bias + nn + j)) : 0.f;
    }

    // This thread's first token of chunk i (nc chunks of each accumulator in turn).
    __device__ __forceinline__ int token(int i) const { return tok0 + 16 * i + (i >= nc ? step1 : 0); }

    static __device__ __forceinline__ uint4 row8(const uint16_t *src, bool vec)
    {
        if (vec)
            return __ldcg(reinterpret_cast<const uint4 *>(src));
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = (uint32_t)__ldcg(src + 2 * j) | ((uint32_t)__ldcg(src + 2 * j + 1) << 16);
        return make_uint4(v[0], v[1], v[2], v[3]);
    }

    // Fetches the operands of chunk i.
    __device__ __forceinline__ void fetch(int i)
    {
        const int m0 = token(i);
        if (nn >= N)
            return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = m0 + 8 * e;
            if (m < M && pmul)
                mul[e] = row8(pmul + (long long)m * ld_mul + nn, vec_mul);
            if (m < M && pres)
                res[e] = row8(pres + (long long)m * ld_res + nn, vec_res);
        }
    }

    // Chunk i from this thread's 16 sums (channel r) to y, its operands fetched
    // before; fetches the next chunk's, if there is one.
    __device__ __forceinline__ void emit(int i, bool next, const float (&v)[16])
    {
        if (out_f32) { // a warp's 32 channels are 128 bytes of a token already
            float *yp = reinterpret_cast<float *>(y);
            const int m0 = token(i) - ot, row = nn - og + r;
            if (row < N)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (m0 + j < M)
                        yp[(size_t)(m0 + j) * N + row] = v[j];
            return;
        }
        float *buf = obuf + ob * (kPfOutB / 4);
        ob ^= 1; // a buffer is written again after the other one's barrier: its readers are through
#pragma unroll
        for (int j = 0; j < 16; ++j)
            buf[j * kPanelRows + r] = v[j];
        named_barrier_sync(id, 128);
        const uint4 cm[2] = {mul[0], mul[1]}, cr[2] = {res[0], res[1]};
        if (next)
            fetch(i + 1);
        const int m0 = token(i);
        if (nn >= N)
            return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = m0 + 8 * e;
            if (m >= M)
                break;
            const float4 a = *reinterpret_cast<const float4 *>(buf + (ot + 8 * e) * kPanelRows + og);
            const float4 b = *reinterpret_cast<const float4 *>(buf + (ot + 8 * e) * kPanelRows + og + 4);
            const size_t at = (size_t)m * N + nn;
            float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] += bias[j];
            epi_activations(x, act);
            const uint32_t mw[4] = {cm[e].x, cm[e].y, cm[e].z, cm[e].w};
            const uint32_t rw[4] = {cr[e].x, cr[e].y, cr[e].z, cr[e].w};
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float m0 = 1.f, m1 = 1.f, r0 = 0.f, r1 = 0.f;
                if (pmul) {
                    m0 = act16_to_float<F16>((uint16_t)mw[j]);
                    m1 = act16_to_float<F16>((uint16_t)(mw[j] >> 16));
                }
                if (pres) {
                    r0 = act16_to_float<F16>((uint16_t)rw[j]);
                    r1 = act16_to_float<F16>((uint16_t)(rw[j] >> 16));
                }
                const float y0 = fmaf(x[2 * j], m0, r0), y1 = fmaf(x[2 * j + 1], m1, r1);
                if constexpr (F16) {
                    const __half2 q2 = __floats2half2_rn(y0, y1);
                    w[j] = *reinterpret_cast<const uint32_t *>(&q2);
                } else {
                    const __nv_bfloat162 q2 = __floats2bfloat162_rn(y0, y1);
                    w[j] = *reinterpret_cast<const uint32_t *>(&q2);
                }
            }
            *reinterpret_cast<uint4 *>(y + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// A tile's sums stand in accumulator b (INT8: in 0 and 1): to y, or, for a tile
// that other pairs share, to this pair's partial and, by the last of them to
// come (a ticket for each CTA's group), added in the pairs' order to y.  The
// accumulators are released after the last column is read.  Called by the four
// warps of a group together.  Out of line, so that the retire loop keeps its
// registers.
template <int BITS, bool F16>
__device__ __noinline__ void pf_flush(const PfParams &p, const PfRetire &rt, int tile, int b)
{
    const int KB = p.KB, lane = threadIdx.x & 31, nc = rt.nc, chunks = nc * p.nsub;
    const uint32_t tq = rt.tq + b * kPfTok;
    const bool whole = rt.u0 <= tile * KB && rt.u1 >= (tile + 1) * KB;
    PfOut<F16> out(p, rt, tile);
    float scale = 1.f;
    const int row = out.nn - out.og + out.r; // the channel whose sums this thread holds
    if (BITS == 8 && row < out.N)
        scale = bf16_bits_to_float(p.scales[row]);
    // pair c's partial of chunk i of this tile
    auto part_of = [&](int c, int i) {
        const int slot = pf_start(p, rt.G, c) / KB == tile ? 0 : 1, sub = i >= rt.nc ? 1 : 0;
        return p.part + (((size_t)((c * 2 + slot) * 2 + rt.rank) * p.nsub + sub) * p.n +
                         16 * (rt.ch0 + i - sub * rt.nc)) * kPanelRows + out.r;
    };
    if (whole)
        out.fetch(0);
    for (int i = 0; i < chunks; ++i) {
        float v[16];
        // The operands and the last chunk's stores branch by lane (ragged N and M): the
        // warp has to be whole again for the tensor-memory load.
        __syncwarp();
        tmem_ld_32x32b_x16(tq + 16 * i + (i >= nc ? kPfTok - 16 * nc : 0), v);
        tmem_wait_ld();
        if (i == chunks - 1) {
            tc_fence_before();
            __syncwarp();
            pf_arrive(rt.ebar + b * 8, lane == 0);
        }
        if (whole) {
            if constexpr (BITS == 8)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] *= scale;
            out.emit(i, i + 1 < chunks, v);
        } else {
            float *mine = part_of(rt.pair, i);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                mine[j * kPanelRows] = v[j];
        }
    }
    if (chunks == 0) { // few tokens: another group has them
        __syncwarp();
        pf_arrive(rt.ebar + b * 8, lane == 0);
    }
    if (whole) {
        __syncwarp();
        return;
    }
    const int cf = pf_owner(p, rt.G, tile * KB), cl = pf_owner(p, rt.G, (tile + 1) * KB - 1);
    uint32_t *counter = p.cnt + (cf * 2 + rt.rank) * PfCfg<BITS>::kGroups + out.id - 1;
    __threadfence();
    named_barrier_sync(out.id, 128);
    if (out.r == 0)
        *rt.ticket = ticket_take_acq_rel(counter);
    named_barrier_sync(out.id, 128);
    const bool last = *rt.ticket == (uint32_t)(cl - cf);
    named_barrier_sync(out.id, 128); // read before the next ticket is written
    if (!last)
        return;
    __threadfence();
    out.fetch(0);
    for (int i = 0; i < chunks; ++i) {
        float t[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            t[j] = 0.f;
        constexpr int CG = 2; // contributors whose loads are in flight together, added in order
        for (int cc = cf; cc <= cl; cc += CG) {
            float v[CG][16];
#pragma unroll
            for (int e = 0; e < CG; ++e)
                if (cc + e <= cl) {
                    const float *src = part_of(cc + e, i);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[e][j] = __ldcg(src + j * kPanelRows);
                }
#pragma unroll
            for (int e = 0; e < CG; ++e)
                if (cc + e <= cl)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        t[j] += v[e][j];
        }
        if constexpr (BITS == 8)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                t[j] *= scale;
        out.emit(i, i + 1 < chunks, t);
    }
    if (out.r == 0)
        atomicExch(counter, 0u); // ready for the next call
    __syncwarp(); // the caller's next tensor-memory instruction is the whole warp's
}

template <int BITS, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PfCfg<BITS>::kThreads, 1)
    gemm_pf_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ PfParams p)
{
    using C = PfCfg<BITS>;
    constexpr int WS = C::kWS, WB = C::kWB, XS = C::kXS, XB = C::kXB, UN = C::kUnroll;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sX = smem;                 // XS x stages, 1024-byte aligned
    uint8_t *sW = sX + XS * XB;         // WS packed blocks
    uint8_t *sO = sW + (size_t)WS * WB;           // two output buffers for each retire group
    uint8_t *sZ = sO + 2 * C::kGroups * kPfOutB;  // WS zero points
    uint64_t *xfull = reinterpret_cast<uint64_t *>(sZ + WS * 128);
    uint64_t *done = xfull + XS;
    uint64_t *afull = done + XS;
    uint64_t *wfull = afull + C::kAS, *wempty = wfull + WS;
    uint64_t *accfull = wempty + WS, *accempty = accfull + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(accempty + 2);
    uint32_t *s_ticket = s_tmem + 1; // [kGroups]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pf_rank();
    const int G = gridDim.x >> 1, pair = blockIdx.x >> 1, KB = p.KB;
    // this pair's units [u0, u1)
    const int u0 = pf_start(p, G, pair), u1 = pf_start(p, G, pair + 1), nu = u1 - u0;
    const int tile0 = u0 / KB, kb0 = u0 % KB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < XS; ++s) {
            mbar_init(&xfull[s], 1); // the leader's expect_tx
            mbar_init(&done[s], 1);
        }
        for (int s = 0; s < WS; ++s) {
            mbar_init(&wfull[s], 1);
            mbar_init(&wempty[s], 8);
        }
        for (int s = 0; s < C::kAS; ++s)
            mbar_init(&afull[s], 16); // the dequantization warps of both CTAs
        for (int s = 0; s < 2; ++s) {
            mbar_init(&accfull[s], 1);
            mbar_init(&accempty[s], 2 * 4 * C::kGroups); // the retire warps of both CTAs
        }
        fence_mbar_init();
    }
    if (warp == 2)
        pf_tmem_alloc(s_tmem);
    if (warp == 0 && lane == 0)
        prefetch_tensormap(&tmx);
    tc_fence_before();
    __syncthreads();
    pf_cluster_sync(); // both CTAs' barriers exist
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *s_tmem;
    bool ok = true;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsIssue));
        if (warp == 0 && lane == 0) {
            // ---------------- x producer ----------------
            pdl_wait(); // x may be written by the preceding kernel
            const uint64_t pol = policy_evict_last();
            const int half = p.n >> 1, tx = p.nsub * p.n * 128; // tx: both CTAs' bytes
            const uint32_t bar = pf_map(xfull, 0);
            int kb = kb0, tt = tile0 % p.TT;
            for (int i = 0; i < 2 * nu; ++i) {
                const int xs = i % XS;
                if (i >= XS && !mbar_wait(&done[xs], ((i / XS) - 1) & 1)) {
                    ok = false;
                    if (rank == 0) // its barriers count both CTAs' bytes
                        pf_landed(xfull, XS, i);
                    break;
                }
                if (rank == 0)
                    mbar_arrive_expect_tx(&xfull[xs], tx);
                for (int sub = 0; sub < p.nsub; ++sub)
                    pf_load_x(sX + xs * XB + sub * kPfXB, &tmx, kb * kBlockK + (i & 1) * 64,
                              (tt * p.nsub + sub) * p.n + (int)rank * half, bar + xs * 8, pol);
                if ((i & 1) && ++kb == KB) {
                    kb = 0;
                    if (++tt == p.TT)
                        tt = 0;
                }
            }
        } else if (warp == 1 && lane == 0) {
            // ---------------- weight producer ----------------
            const uint64_t pol = policy_evict_first();
            int kb = kb0, tt = tile0 % p.TT, pnl = 2 * (tile0 / p.TT) + (int)rank;
            int ws = 0;
            uint32_t wpar = 1; // the stage's last round; its first needs no wait
            for (int i = 0; i < nu; ++i) {
                if (i >= WS && !mbar_wait(&wempty[ws], wpar)) {
                    ok = false;
                    pf_landed(wfull, WS, i);
                    break;
                }
                const size_t blk = (size_t)pnl * KB + kb;
                if (pnl < p.panels) {
                    mbar_arrive_expect_tx(&wfull[ws], WB + (BITS == 4 ? 64 : 0));
                    bulk_g2s(sW + (size_t)ws * WB, p.wq + blk * WB, WB, &wfull[ws], pol);
                    if constexpr (BITS == 4)
                        bulk_g2s(sZ + ws * 128, p.zeros + blk * 64, 64, &wfull[ws], pol);
                } else {
                    mbar_arrive(&wfull[ws]); // no such panel: its rows are never written
                }
                if (++ws == WS) {
                    ws = 0;
                    wpar ^= 1;
                }
                if (++kb == KB) {
                    kb = 0;
                    if (++tt == p.TT) {
                        tt = 0;
                        pnl += 2;
                    }
                }
            }
        } else if (warp == 2 && rank == 0) {
            // ---------------- MMA issuer ----------------
            // The whole warp walks the steps, so that addresses and descriptors
            // stay in uniform registers; one lane issues.  Unrolled over the ring,
            // whose slots, stages and parities are then constants: the loop's own
            // instructions cost as much as the products otherwise.
            const bool issuer = pf_elect();
            const uint32_t idesc = (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(p.n >> 3) << 17) | (16u << 24);
            const uint64_t bdesc0 = smem_desc_sw128(smem_u32(sX));
            int kb = kb0, tiles = 0; // tiles begun (INT8)
            uint32_t par = 0;        // of this round of the x ring
            for (int i0 = 0; i0 < nu && ok; i0 += UN, par ^= 1) {
#pragma unroll
                for (int uu = 0; uu < UN; ++uu) {
                    if (i0 + uu >= nu)
                        break;
                    const int as = uu & 1; // INT8: A stage; INT4: accumulator
                    bool fresh = true;
                    if constexpr (BITS == 8) {
                        fresh = kb == 0 || i0 + uu == 0;
                        // the last tile's sums must have been read
                        if (fresh && ++tiles > 1)
                            ok = ok && mbar_wait(&accempty[0], tiles & 1);
                        ok = ok && mbar_wait(&afull[as], par);
                    } else { // group g = i0 + uu waits for the release of g - 2
                        if (i0 > 0 || uu >= 2)
                            ok = ok && mbar_wait(&accempty[as], ((uu >> 1) + 1) & 1);
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int j = 2 * uu + hf;
                        if constexpr (BITS == 4) // step 8 (round) + j: the stage's use j / 4 of the round's two
                            ok = ok && mbar_wait(&afull[j % 4], (j >> 2) & 1);
                        ok = ok && mbar_wait(&xfull[j], par);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (issuer) {
                            const uint64_t bdesc = bdesc0 + (uint64_t)(j * (XB >> 4));
                            const uint32_t d = tmem + (BITS == 4 ? as * kPfTok : 0);
                            const uint32_t a = tmem + kPfA0 + (j % 4) * 32;
                            const uint32_t keep = fresh && hf == 0 ? 0u : 1u;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                pf_mma(d, a + kk * 8, bdesc + (uint64_t)(kk * 2), idesc, kk == 0 ? keep : 1u);
                            if (BITS == 8 && p.nsub == 2)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    pf_mma(d + kPfTok, a + kk * 8, bdesc + (uint64_t)((kPfXB >> 4) + kk * 2), idesc,
                                           kk == 0 ? keep : 1u);
                            pf_commit(&done[j]);
                        }
                        __syncwarp();
                    }
                    if (!ok)
                        break;
                    if (++kb == KB)
                        kb = 0;
                    if (BITS == 8 && (kb == 0 || i0 + uu == nu - 1) && issuer)
                        pf_commit(&accfull[0]);
                    __syncwarp();
                }
            }
        }
    } else if (warp < 4 + 4 * C::kGroups) {
        // ---------------- retire warps ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsRetire));
        pdl_wait(); // y and the workspace may still be in use by the preceding kernel
        const int q = warp & 3, h = (warp - 4) >> 2;
        const int nch = p.n / 16;
        static_assert(C::kGroups * C::kChunks * 16 == kPfTok, "the groups cover an accumulator");
        PfRetire rt;
        rt.ch0 = nch * h / C::kGroups; // this warp's 16-column chunks
        rt.nc = nch * (h + 1) / C::kGroups - rt.ch0;
        rt.G = G;
        rt.pair = pair;
        rt.rank = (int)rank;
        rt.u0 = u0;
        rt.u1 = u1;
        rt.obuf = reinterpret_cast<float *>(sO) + h * 2 * (kPfOutB / 4);
        rt.ticket = s_ticket + h;
        rt.ebar = pf_map(accempty, 0);
        rt.tq = tmem + ((uint32_t)(32 * q) << 16) + 16 * rt.ch0;
        const int r = 32 * q + lane, nc = rt.nc;
        const uint32_t tq = rt.tq;

        if constexpr (BITS == 4) {
            unsigned long long tot[C::kChunks * 8]; // pairs of fp32 sums
#pragma unroll
            for (int j = 0; j < C::kChunks * 8; ++j)
                tot[j] = 0ull;
            int tile = tile0, kb = kb0;
            // this thread's scales, two groups ahead of their use within a tile
            const uint16_t *sp;
            uint16_t sc0, sc1;
            auto scales_of = [&]() { // of (tile, kb) and the group after it
                const int pnl = min(2 * (tile / p.TT) + (int)rank, p.panels - 1); // a panel past the last is never written
                sp = p.scales + ((size_t)pnl * KB + kb) * kPanelRows + r;
                sc0 = __ldg(sp);
                sc1 = kb + 1 < KB ? __ldg(sp + kPanelRows) : 0;
            };
            scales_of();
            for (int g = 0; g < nu; ++g) {
                const int st = 2 * g + 1; // the group's last step
                const float s = bf16_bits_to_float(sc0);
                sc0 = sc1;
                if (kb + 2 < KB)
                    sc1 = __ldg(sp + 2 * kPanelRows);
                sp += kPanelRows;
                ++kb;
                bool end = kb == KB || g == nu - 1;
                // A warp whose wait gave up goes on without waiting, so that every
                // warp of the group comes to the barriers of every tile.
                ok = ok && mbar_wait_warp(&done[st % XS], (st / XS) & 1);
                tc_fence_after();
                unsigned long long s2;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
                const uint32_t ta = tq + (g & 1) * kPfTok;
#pragma unroll
                for (int c = 0; c < C::kChunks; c += 2) { // two loads in flight; columns past the group's are not used
                    float v[2][16];
                    tmem_ld_32x32b_x16(ta + 16 * c, v[0]);
                    tmem_ld_32x32b_x16(ta + 16 * c + 16, v[1]);
                    tmem_wait_ld();
                    if (c + 2 == C::kChunks) { // every column is read: released before the last are used
                        tc_fence_before();
                        __syncwarp();
                        pf_arrive(rt.ebar + (g & 1) * 8, lane == 0 && !end);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
                            pf_ffma2(tot[8 * (c + e) + j / 2], s2, v[e][j], v[e][j + 1]);
                }
                if (!end)
                    continue;
                // the tile's (or the run's) last group: the totals take its
                // accumulator's place, so that writing them out needs few registers
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                    if (c < nc) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            w[2 * j] = (uint32_t)tot[8 * c + j];
                            w[2 * j + 1] = (uint32_t)(tot[8 * c + j] >> 32);
                        }
                        tmem_st_32x32b_x16(ta + 16 * c, w);
                    }
                tmem_wait_st();
                ok = pf_all(1 + h, ok);
                if (ok)
                    pf_flush<BITS, F16>(p, rt, tile, g & 1);
#pragma unroll
                for (int j = 0; j < C::kChunks * 8; ++j)
                    tot[j] = 0ull;
                kb = 0;
                ++tile;
                if (g < nu - 1)
                    scales_of();
            }
        } else {
            const int tile1 = nu > 0 ? (u1 - 1) / KB : tile0 - 1;
            for (int tile = tile0; tile <= tile1; ++tile) {
                ok = pf_all(1 + h, ok && mbar_wait_warp(&accfull[0], (tile - tile0) & 1));
                if (!ok)
                    break; // the whole group
                tc_fence_after();
                pf_flush<BITS, F16>(p, rt, tile, 0);
            }
        }
    } else {
        // ---------------- dequantization warps ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsDequant));
        const int q = warp & 3, e = (warp - 4 - 4 * C::kGroups) >> 2;
        const uint32_t bar = pf_map(afull, 0);
        const int r = 32 * q + lane, g = lane >> 2, blkrow = 2 * q + e; // INT8: this lane's row; INT4: 16-row block
        constexpr int AH = C::kAH, V = BITS == 4 ? 1 : 2; // V: 16-byte pieces of 64 k
        uint4 w[AH * V];                                  // this lane's packed values of an A stage
        uint32_t zlo = 0, zhi = 0;
        int ws = 0;
        uint32_t wpar = 0;
        auto fetch = [&](int h0) { // halves h0 .. h0 + AH - 1 of weight stage ws
            const uint8_t *blk = sW + (size_t)ws * WB;
#pragma unroll
            for (int hf = 0; hf < AH; ++hf) {
                if constexpr (BITS == 4) {
                    w[hf] = *reinterpret_cast<const uint4 *>(blk + blkrow * 1024 + (h0 + hf) * 512 + lane * 16);
                } else {
                    const int c = 4 * (h0 + hf) + 2 * e; // two 16-k chunks of one row
                    w[2 * hf] = *reinterpret_cast<const uint4 *>(blk + int8_chunk_in_block(r, c));
                    w[2 * hf + 1] = *reinterpret_cast<const uint4 *>(blk + int8_chunk_in_block(r, c + 1));
                }
            }
            if (BITS == 4 && h0 == 0) { // rows 16 blkrow + g and + 8
                const uint8_t *zp = sZ + ws * 128 + 8 * blkrow + (g >> 1);
                const uint32_t z0 = (zp[0] >> (4 * (g & 1))) & 0xFu, z1 = (zp[4] >> (4 * (g & 1))) & 0xFu;
                zlo = kPfMagic2<F16> | z0 | (z0 << 16);
                zhi = kPfMagic2<F16> | z1 | (z1 << 16);
            }
        };
        ok = mbar_wait_warp(&wfull[0], 0);
        if (ok)
            fetch(0);
        // stages of a round of the x ring: INT4 eight of one half, INT8 two of two
        constexpr int RS = XS / AH;
        const int stages = 2 * nu / AH;
        uint32_t par = 0; // of this round
        for (int i0 = 0; i0 < stages && ok; i0 += RS, par ^= 1) {
#pragma unroll
            for (int j = 0; j < RS; ++j) {
                if (i0 + j >= stages)
                    break;
                uint32_t rr[AH][16];
#pragma unroll
                for (int hf = 0; hf < AH; ++hf) {
                    if constexpr (BITS == 4) {
                        pf_int4_regs<F16>(w[hf], zlo, zhi, rr[hf]);
                    } else {
                        const uint4 a = w[2 * hf], b = w[2 * hf + 1];
                        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            rr[hf][2 * i] = pf_s8pair<F16>(v[i], 0);
                            rr[hf][2 * i + 1] = pf_s8pair<F16>(v[i], 1);
                        }
                    }
                }
                // the next stage's values, before this one's wait for its place
                if (AH == 1 && (j & 1) == 0) {
                    fetch(1);
                } else { // every value loaded from the weight stage has been used: release it
                    __syncwarp();
                    pf_arrive_own(&wempty[ws], lane == 0);
                    if (++ws == WS) {
                        ws = 0;
                        wpar ^= 1;
                    }
                    if (i0 + j + 1 < stages) {
                        if (!mbar_wait_warp(&wfull[ws], wpar)) {
                            ok = false;
                            break;
                        }
                        fetch(0);
                    }
                }
                // the A stage's last products: four halves back, in this round of
                // the ring or (its first kAS stages) the last
                const bool same = j >= C::kAS;
                const int slot = ((j - C::kAS) * AH + AH - 1 + XS) % XS;
                if ((i0 > 0 || same) && !mbar_wait_warp(&done[slot], same ? par : par ^ 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = tmem + kPfA0 + (j % C::kAS) * AH * 32 + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int hf = 0; hf < AH; ++hf) {
                    if constexpr (BITS == 4)
                        tmem_st_16x256b_x4(ta + ((uint32_t)(16 * e) << 16) + 32 * hf, rr[hf]);
                    else
                        tmem_st_32x32b_x16(ta + 32 * hf + 16 * e, rr[hf]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                pf_arrive(bar + (j % C::kAS) * 8, lane == 0);
            }
        }
    }

    if (!ok)
        atomicExch(&g_gemm_pf_error, kErrTimeout);
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    pf_cluster_sync(); // neither CTA leaves while the other may still signal it
    if (warp == 2) {
        tc_fence_after();
        pf_tmem_dealloc(tmem);
    }
}

bool pf_x_map(CUtensorMap *map, const uint16_t *x, int M, int K, int rows)
{
    auto fn = get_encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M};
    const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a launch is cut: tokens of an accumulator, accumulators and tiles, pairs of
// CTAs, whole tiles or equal runs of units.
struct PfPlan {
    int n, nsub, TT, G, align;
};

// The cheapest of a few cuts, by times measured on B200 (us): a unit takes
// 0.87 (INT4; its retirement, whatever the tokens) or 0.5 + 0.0018 a token
// (INT8; dequantization, then the products), a tile 0.3 a 16-token chunk of its
// two retire groups to write out, and cutting tiles between pairs 8 at once and 0.3 a
// chunk for the partial sums and for each pair.  Many tokens a tile share a
// dequantized block; more tiles keep all pairs busy without cutting them.
PfPlan pf_plan(int bits, int M, int panels, int KB, int pairs, size_t ws_bytes)
{
    PfPlan best{0, 0, 0, 0, 1};
    double best_us = 0;
    const int pp = (panels + 1) / 2, sub = bits == 8 ? 2 : 1;
    for (int nsub = 1; nsub <= (M <= kPfTok ? 1 : sub); ++nsub) {
        for (int cut = 1; cut <= 6; ++cut) { // tiles of a channel panel pair: as few as hold the tokens, times cut
            PfPlan q;
            q.nsub = nsub;
            const int least = (M + nsub * kPfTok - 1) / (nsub * kPfTok), most = (M + 16 * nsub - 1) / (16 * nsub);
            const int want = least * cut < most ? least * cut : most;
            q.n = ((M + want * nsub - 1) / (want * nsub) + 15) / 16 * 16;
            q.TT = (M + nsub * q.n - 1) / (nsub * q.n);
            const long long tiles = (long long)pp * q.TT, units = tiles * KB;
            if (units >= (1LL << 31))
                break;
            const double tok = q.n * q.nsub, chunks = tok / 32;
            const double unit = bits == 8 ? 0.5 + 0.0018 * tok : 0.87, out = 0.3 * chunks;
            auto consider = [&](int G, int align, double us) {
                if (best.G == 0 || us < best_us) {
                    best_us = us;
                    best = q;
                    best.G = G;
                    best.align = align;
                }
            };
            const long long rounds = (tiles + pairs - 1) / pairs;
            consider((int)(tiles < pairs ? tiles : pairs), 1, rounds * (KB * unit + out));
            // equal runs: every pair, or a whole number of pairs a tile
            for (int c = 2; c <= 8; ++c) {
                const long long G = c == 8 ? pairs : tiles * c;
                if (G > pairs || units < 4 * G) // a run of less than 512 k is not worth its partial sums
                    continue;
                if (ws_bytes < ws_counter_bytes() + (size_t)G * 4 * q.nsub * q.n * kPanelRows * sizeof(float))
                    continue;
                const double run = (double)units / G, parts = run >= KB ? 2 : KB / run + (c == 8 ? 1 : 0);
                consider((int)G, 0,
                         8 + run * unit + (run / KB + 1) * out + chunks * (0.3 + 0.3 * parts));
            }
        }
    }
    return best;
}

template <int BITS, bool F16>
cudaError_t launch_pf_t(const LinearArgs &a, void *ws, size_t ws_bytes, int sm_count, cudaStream_t st)
{
    constexpr size_t smem = pf_smem_bytes<BITS>();
    static_assert(smem <= 227 * 1024, "shared memory per CTA");
    cudaError_t e = kernel_setup((const void *)gemm_pf_kernel<BITS, F16>, smem, 0, 0, nullptr);
    if (e != cudaSuccess)
        return e;
    // the warps' shares after setmaxnreg must fit what the CTA is launched with,
    // or the retire warps would wait for registers that never come
    static std::atomic<int> known{0}; // the same on every device
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, (const void *)gemm_pf_kernel<BITS, F16>)) != cudaSuccess)
            return e;
        regs = fa.numRegs;
        known.store(regs, std::memory_order_relaxed);
    }
    if (regs * PfCfg<BITS>::kThreads < PfCfg<BITS>::kRegs)
        return cudaErrorInvalidConfiguration;
    const Shape sh{a.bits, a.K, a.N, a.group};
    PfParams p;
    p.M = a.M;
    p.N = a.N;
    p.KB = sh.kblocks();
    p.panels = sh.panels();
    const int pairs = sm_count / 2 < kPfMaxPairs ? sm_count / 2 : kPfMaxPairs;
    const PfPlan plan = pf_plan(BITS, a.M, p.panels, p.KB, pairs, ws_bytes);
    if (plan.G == 0)
        return cudaErrorInvalidValue; // the caller cuts M (pf_max_tokens)
    p.nsub = plan.nsub;
    p.n = plan.n;
    p.TT = plan.TT;
    p.tiles = (p.panels + 1) / 2 * p.TT;
    p.U = p.tiles * p.KB;
    p.align = plan.align;
    const int G = plan.G;
    p.wq = (const uint8_t *)a.wq;
    p.scales = (const uint16_t *)a.scales;
    p.zeros = (const uint8_t *)a.zeros;
    p.y = a.y;
    p.epi = *a.epi;
    p.cnt = (uint32_t *)ws;
    p.part = ws ? (float *)((uint8_t *)ws + ws_counter_bytes()) : nullptr;
    CUtensorMap map;
    if (!pf_x_map(&map, a.x, a.M, a.K, p.n / 2))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2 * G);
    cfg.blockDim = dim3(PfCfg<BITS>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, gemm_pf_kernel<BITS, F16>, map, p);
}

} // namespace

void pf_plan_debug(int bits, int M, int K, int N, int pairs, size_t ws_bytes, int *plan)
{
    const PfPlan q = pf_plan(bits, M, (N + kPanelRows - 1) / kPanelRows, (K + kBlockK - 1) / kBlockK,
                             pairs < kPfMaxPairs ? pairs : kPfMaxPairs, ws_bytes);
    const int v[5] = {q.n, q.nsub, q.TT, q.G, q.align};
    for (int i = 0; i < 5; ++i)
        plan[i] = v[i];
}

// Tokens of one launch: its units stay below 2^31.
int pf_max_tokens(int K, int N)
{
    const long long per_tile = (long long)((N + 255) / 256) * ((K + kBlockK - 1) / kBlockK);
    const long long t = ((1LL << 31) - 1) / per_tile * kPfTok;
    return t > kMaxTokens ? kMaxTokens : (int)t;
}

cudaError_t launch_gemm_pf(const LinearArgs &a, void *ws, size_t ws_bytes, int sm_count, cudaStream_t st, bool f16)
{
    const size_t have = ws ? ws_bytes : 0;
    if (f16)
        return a.bits == 8 ? launch_pf_t<8, true>(a, ws, have, sm_count, st)
                           : launch_pf_t<4, true>(a, ws, have, sm_count, st);
    return a.bits == 8 ? launch_pf_t<8, false>(a, ws, have, sm_count, st)
                       : launch_pf_t<4, false>(a, ws, have, sm_count, st);
}

cudaError_t read_gemm_pf_error(int *code, cudaStream_t st)
{
    int host = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&host, g_gemm_pf_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess)
        return e;
    e = cudaMemcpyToSymbolAsync(g_gemm_pf_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess)
        return e;
    e = cudaStreamSynchronize(st);
    *code = host;
    return e;
}

} // namespace wq
