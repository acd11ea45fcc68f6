// paged_chunk.cu - attention of chunks of new tokens over a paged key/value
// cache on the 5th-generation tensor cores (sm_103a).  Formulas, plan and the
// merge of partial results: paged_attend.cu.
//
// Both products are matrix products with enough rows to fill the tensor cores,
// so they bound the kernel.  An item is 256 query rows of one kv head (all GQ
// query heads of up to 2 * floor(128 / GQ) tokens, so a key tile is read once
// for all of them) against a run of 128-key tiles, in two tiles of 128 rows
// that share every key and value tile.  Tensor memory holds one score tile
// (128 columns), the weights of both tiles as 16-bit pairs (2 x 64) and both
// outputs (2 x 128): a score tile is copied to registers as soon as it is there
// and its place goes to the other tile's next scores, so that the next product
// never waits for a softmax (with a score tile of its own each, whose place the
// weights took over, the chain scores - softmax - values - next scores bound the
// kernel: 1.98 us for two tiles of 128 x 128, of which the products are 1.07).
// Scores and weights never leave the SM.
//
// Roles (one CTA per SM): two groups of 4 softmax warps, a thread per query
// row; one warp that streams queries, keys and values by TMA (a box per page);
// two warps that issue tcgen05.mma, one for scores, one for values.  With an
// 8-bit cache eight more warps turn the codes into fp16 operands in shared
// memory (4096 bf16 queries over 16384 keys: four took 815 us, eight 763).
//
// What bounds it (that chunk over a 16-bit cache: 675 us, 1.42 PFLOP/s, where the
// inputs change from call to call, 627 on one set of tensors; over codes, on one
// set, 807): a pair of tiles takes 1.5 us where the products take 1.07.  The
// score tile waits for its copy to registers between products, and by its bytes
// (192 KB of operands read, 64 KB copied in) shared memory is as busy as the
// tensor core.  Over codes the softmax warps have 176 registers instead of 208,
// and 20 warps of four kinds of code share the instruction caches.  A run of an
// item takes about 4 us besides its tiles (6 over codes): its first keys' way
// through the pipeline and its output's to memory.
//
// 8-bit cache.  A factor per key inside the softmax (2 x 128 numbers a tile to
// every thread) cost more than the softmax itself.  So the exponents are split
// in a tile's largest among the keys that are seen, A of keys and B of values,
// and each key's rest:
// the operands are code * 2^(a - A) and code * 2^(b - B), and a tile's two
// exponents act once per score: t = scale 2^A (q . K') + B, w = 2^(t - M) with M
// the running maximum of t, out = sum w V' / sum w 2^-B.  That holds while the
// seen keys of a tile have exponents within KEYS_WITHIN and values within
// VALUES_WITHIN of the largest.  Codes are multiples of 2^-9, so the operands are
// exact in fp16 down to 2^-15 of the largest row; and M lies at most 2^8 above
// what some seen value asks for, so that a row's largest w 2^b is at least 2^-1
// and its weights keep all of fp16's bits down to 2^-13 of that.  A tile whose
// exponents lie further apart (its one exponent would be that of a row which may
// have no weight at all) takes the codes as they are, and the exponents act key
// by key in the softmax, as for single tokens:
// t_j = scale 2^a_j (q . K_j) + b_j, and sum w_j 2^-b_j below the line.  So does a
// tile with zero value rows: those count with the least exponent, which their
// codes have to be read for.
// Operands are fp16 whatever the queries' type, since one instruction makes them
// of two codes (bf16 takes five: 996 us against 884 for the chunk above, with
// four warps); bf16 queries become fp16 by a power of two for each row, in place,
// while the output of the item before is still to be written.
//
// The output is rescaled only when a row's maximum grew by more than 2^LAG
// (the softmax warps do it in tensor memory between two products), so weights
// reach up to 2^(OFF + LAG) and nearly no tile pays for it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "tcgen05.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pk_err);

constexpr int D = 128;
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float OFF = 7.0f, LAG = 8.0f;
constexpr int KEYS_WITHIN = 15, VALUES_WITHIN = 8;  // powers of two that rows of a tile may share an exponent over
constexpr int TILE_B = PG_TILE * D * 2;  // a 16-bit tile of 128 rows: two halves of 64 columns
constexpr int HALF_B = TILE_B / 2;
constexpr int RAW_B = PG_TILE * D;       // a tile of codes

template <bool Q8> struct CkShape {
    static constexpr int STAGES = Q8 ? 3 : 4;   // 16-bit key / value tiles
    static constexpr int RAW = Q8 ? 3 : 0;      // tiles of codes in flight
    static constexpr int META = Q8 ? 2 : 0;     // key tiles whose exponents are unpacked
    static constexpr int CONV = Q8 ? 8 : 0;     // warps that convert codes
    static constexpr int WARPS = 12 + CONV;
    static constexpr int THREADS = 32 * WARPS;
    // registers a thread: at launch, the softmax warps, warps 8-11, the converting
    // warps; the shares of all warps add up to the launch's at most
    static constexpr int REGS = Q8 ? 96 : 168, R_SOFT = Q8 ? 176 : 208, R_CTL = Q8 ? 48 : 88, R_CONV = 40;
    static_assert(256 * R_SOFT + 128 * R_CTL + 32 * CONV * R_CONV <= THREADS * REGS, "registers of one CTA");
    static constexpr int BARS = 3 + 2 * STAGES + 7 + 2 * RAW + 2 * META + 2;
    static constexpr int RUNS = 8 * 64;         // the softmax warps' runs
    static constexpr int SMEM = 1024 + 2 * TILE_B + STAGES * TILE_B + RAW * RAW_B + RUNS + RAW * 2 * PG_TILE +
                                RAW * 32 + META * (16 + 8 * PG_TILE) + 8 * (Q8 ? 2 : 1) * BARS + 16;
};
static_assert(CkShape<false>::SMEM <= 232448 && CkShape<true>::SMEM <= 232448, "shared memory of one CTA");

constexpr uint32_t CK_TIMEOUT = 1, CK_BY_KEY = 2;  // why every role stops

template <bool Q8> struct CkBars {
    using C = CkShape<Q8>;
    uint64_t *q_full, *q_empty, *kv_full, *kv_empty, *s_full, *p_full, *pv_done, *s_free, *raw_full, *raw_empty, *meta_full,
        *meta_empty, *drain, *q_ready;
    __device__ __forceinline__ explicit CkBars(uint64_t *b)
        : q_full(b), q_empty(b + 1), kv_full(b + 2), kv_empty(kv_full + C::STAGES), s_full(kv_empty + C::STAGES),
          p_full(s_full + 2), pv_done(p_full + 2), s_free(pv_done + 2), raw_full(s_free + 1), raw_empty(raw_full + C::RAW),
          meta_full(raw_empty + C::RAW), meta_empty(meta_full + C::META), drain(meta_empty + C::META), q_ready(drain + 2)
    {
    }
    __device__ __forceinline__ void init()
    {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&kv_full[s], Q8 ? C::CONV : 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&s_full[w], 1);
            mbar_init(&p_full[w], 4);
            mbar_init(&pv_done[w], 1);
        }
        mbar_init(s_free, 4);
        for (int s = 0; s < C::RAW; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], C::CONV);
        }
        for (int s = 0; s < C::META; ++s) {
            mbar_init(&meta_full[s], C::CONV);
            mbar_init(&meta_empty[s], 8);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        mbar_init(q_ready, 8);
    }
};

// Operand B of the value product: rows are keys (K), 64-column halves side by
// side (N contiguous): 128-byte swizzle, 8-key groups 1024 bytes apart, the
// halves HALF_B apart.
__device__ __forceinline__ uint64_t ck_desc_v(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(HALF_B >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor: fp32 accumulator, M = N = 128, both operands fp16 or
// both bf16; `b_mn`: B has its N dimension contiguous.
__host__ __device__ constexpr uint32_t ck_idesc(bool bf16, bool b_mn)
{
    return qt_idesc(128) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u);
}

// The products of one 128 x 128 x 128 tile, eight K = 16 steps, by one elected
// thread of the (whole, converged) warp.  One block of PTX each, so that the
// operands' addresses stay in uniform registers: issued one by one from a
// branch on the lane number, an instruction took 107 cycles to issue where the
// tensor core needs 64.  `bar` (shared) gets an arrival when they are done.

// D = A B, both from shared memory, rows of 64 entries: steps 32 bytes apart,
// the second half of K HALF_B further.
__device__ __forceinline__ void ck_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t bar)
{
    static_assert(HALF_B == 16384, "the descriptors' steps below");
    asm volatile(
        "{\n\t.reg .pred q, f, t;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 t, 1, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
        "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 1024;\n\t"
        "add.s64 b5, %2, 1026;\n\tadd.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(bar)
        : "memory");
}

// D (+)= A B with A (16-bit pairs) in tensor memory, 8 columns a step, and B's
// rows (keys) 2048 bytes a step; acc 0: D is overwritten.
__device__ __forceinline__ void ck_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q, f, t;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t"
        ".reg .b64 b1, b2, b3, b4, b5, b6, b7;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 t, 1, 0;\n\tsetp.ne.b32 f, %4, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\tadd.s32 a4, %1, 32;\n\t"
        "add.s32 a5, %1, 40;\n\tadd.s32 a6, %1, 48;\n\tadd.s32 a7, %1, 56;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\tadd.s64 b4, %2, 512;\n\t"
        "add.s64 b5, %2, 640;\n\tadd.s64 b6, %2, 768;\n\tadd.s64 b7, %2, 896;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(bar)
        : "memory");
}

// An arrival on `bar` when every product that this warp's elected thread issued
// is done.
__device__ __forceinline__ void ck_commit(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void ck_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void ck_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// L2 policy of the cache's tiles: other CTAs read them too.
__device__ __forceinline__ uint64_t ck_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// 16 consecutive fp32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void ck_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void ck_hold16(uint32_t (&r)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(r[j])::"memory");
}

__device__ __forceinline__ float2 ck_f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// A word with its n lowest bits set (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t ck_below(int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; }

template <int N> __device__ __forceinline__ void ck_reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void ck_reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <class T> __device__ __forceinline__ uint32_t ck_pack(float a, float b);
template <> __device__ __forceinline__ uint32_t ck_pack<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t ck_pack<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^e twice in fp16, -15 <= e <= 0; of a key that nothing sees e may be any number.
__device__ __forceinline__ uint32_t ck_factor(int e)
{
    static_assert(KEYS_WITHIN <= 15 && VALUES_WITHIN <= 15, "factors of seen keys");
    return 0x00010001u * (e >= -14 ? (uint32_t)(min(e, 0) + 15) << 10 : 1u << 9);
}

// Four codes times a factor as two pairs of fp16.
__device__ __forceinline__ void ck_operand(uint32_t four, uint32_t f, uint32_t &lo, uint32_t &hi)
{
    uint32_t a, b;
    e4m3x4_to_f16x4(four, a, b);
    const __half2 g = *reinterpret_cast<const __half2 *>(&f);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&a), g), y = __hmul2(*reinterpret_cast<const __half2 *>(&b), g);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// One row of a bf16 query tile becomes fp16, by a power of two that brings its
// largest entry to [2^14, 2^15): exact but for entries 2^-28 of that and below.
// Returns the power that undoes it.
__device__ __forceinline__ float ck_query(unsigned char *tile, int row)
{
    uint32_t top = 0u;
#pragma unroll 8
    for (int c = 0; c < 16; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * HALF_B + swz128(row, c & 7));
        top = __vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    const int e = max((int)(max(top & 0xffffu, top >> 16) >> 7) - 127, -100);
    const float f = pow2f(14 - e);
#pragma unroll 4
    for (int c = 0; c < 16; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(tile + (c >> 3) * HALF_B + swz128(row, c & 7));
        uint4 v = *at;
        auto one = [&](uint32_t &x) {
            const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
            x = ck_pack<__half>(a.x * f, a.y * f);
        };
        one(v.x);
        one(v.y);
        one(v.z);
        one(v.w);
        *at = v;
    }
    return pow2f(e - 14);
}

// A softmax warp keeps its run in shared memory and reads it where it needs it:
// what it held in registers beside the scores went to local memory, and after
// the output's stores came back from L2 1.6 us later.
__device__ __forceinline__ PgRun ck_run(uint32_t at)
{
    int v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                     : "r"(at + 16 * i)
                     : "memory");
    PgRun r;
    r.e.b = v[0]; r.e.tok0 = v[1]; r.e.nt = v[2]; r.e.p0 = v[3];
    r.e.hi = v[4]; r.e.nsink = v[5]; r.e.tl = v[6]; r.e.ntiles = v[7];
    r.ei = v[8]; r.h = v[9]; r.t0 = v[10]; r.tn = v[11];
    r.left = v[12]; r.first = v[13] != 0;
    return r;
}
// The run of the softmax warp that is furthest behind.
__device__ __forceinline__ PgRun ck_run_behind(const unsigned char *srun)
{
    auto left = [&](int w) { return reinterpret_cast<const volatile int *>(srun + 64 * w)[12]; };
    int b = 0;
#pragma unroll 1
    for (int w = 1; w < 8; ++w)
        if (left(w) > left(b)) b = w;
    return ck_run(smem_u32(srun + 64 * b));
}
__device__ __forceinline__ void ck_keep(uint32_t at, const PgRun &r, int lane)
{
    __syncwarp();
    if (lane == 0) {
        const int v[16] = {r.e.b, r.e.tok0, r.e.nt, r.e.p0, r.e.hi, r.e.nsink, r.e.tl, r.e.ntiles,
                           r.ei, r.h, r.t0, r.tn, r.left, (int)r.first, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * i), "r"(v[4 * i]), "r"(v[4 * i + 1]),
                         "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                         : "memory");
    }
    __syncwarp();
}

// 32 bytes to an address that is a multiple of 32.
__device__ __forceinline__ void ck_store32(void *at, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Largest of the bytes that the lanes of a warp hold.
__device__ __forceinline__ int ck_top(uint32_t four)
{
    four = __vmaxu4(four, four >> 16);
    return (int)__reduce_max_sync(FULL_MASK, max(four & 0xffu, (four >> 8) & 0xffu));
}

// 255 in the bytes that are below `least`.
__device__ __forceinline__ uint32_t ck_less(uint32_t four, int least)
{
    return __vcmpltu4(four, 0x01010101u * (uint32_t)max(least, 0));
}

template <class T, bool Q8>
__global__ void __launch_bounds__(CkShape<Q8>::THREADS, 1) paged_chunk_kernel(const __grid_constant__ PagedAttendParams p)
{
    using C = CkShape<Q8>;
    using TV = typename std::conditional<Q8, __half, T>::type;  // of both products' operands
    constexpr int STAGES = C::STAGES;
    constexpr bool BFV = std::is_same<TV, __nv_bfloat16>::value;
    constexpr bool QC = !std::is_same<T, TV>::value;  // queries are converted
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *sq = smem_1k(smem_raw);                  // two query tiles
    unsigned char *skv = sq + 2 * TILE_B;                   // key / value tiles
    unsigned char *sraw = skv + STAGES * TILE_B;            // tiles of codes
    unsigned char *srun = sraw + C::RAW * RAW_B;            // [8][64] the softmax warps' runs
    unsigned char *sexp = srun + C::RUNS;                   // [RAW][2][128] exponents (of key tiles)
    float4 *smeta = reinterpret_cast<float4 *>(sexp + C::RAW * 2 * PG_TILE);  // [META] |scale| 2^A, B, 2^-B, 1: key by key
    float4 *skeys = smeta + C::META;                        // [META][128] |scale| 2^a, b of a tile taken key by key
    int *srow = reinterpret_cast<int *>(skeys + C::META * (PG_TILE / 2));     // [RAW][8] rows of a key tile's boxes
    uint64_t *bars = reinterpret_cast<uint64_t *>(srow + C::RAW * 8);
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(bars + (Q8 ? 2 : 1) * C::BARS);
    volatile uint32_t *abort_flag = tslot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tqt = 128 / p.GQ;  // tokens of one query tile
    if (threadIdx.x == 0) {
        CkBars<Q8>(bars).init();
        if constexpr (Q8) CkBars<Q8>(bars + C::BARS).init();
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(const_cast<uint32_t *>(tslot), 512);
    pg_wait();  // for the plan
    pg_go();
    PgRun r_all;
    r_all.start(p.large.start[blockIdx.x]);
    qt_fence_before();
    __syncthreads();
    qt_fence_after();
    if (r_all.left <= 0) {  // the whole CTA
        if (warp == 9) tmem_free(*tslot, 512);
        return;
    }
    const uint32_t tmem = *tslot;  // scores at 0, weights at 128 and 192, outputs at 256 and 384

    // Bounded wait; gives up (and makes every role give up) after the limit.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > MBAR_TIMEOUT_NS) {
                atomicOr(&g_pk_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
                *abort_flag = CK_TIMEOUT;
                return false;
            }
        }
    };

    // A role goes through the CTA's share.  Over codes, the converting warps end
    // that at the first tile whose exponents lie too far apart or that may have
    // zero value rows, and the CTA goes on from that item's run with roles that can
    // take the exponents key by key.  One body for both took 10 to 18 % longer on
    // every tile, since softmax and converting warps have no register or instruction
    // to spare; the check in a warp of its own 14 %, in the copying warp 6 to 14 %.
    // So it is 1 to 4 % (4096 queries over 16384 keys: fp16 805 us against 801
    // without the check, bf16 807 against 779), and that call takes 1.2 ms where
    // token 0 has a zero value row, 1.1 where values reach beyond 224 (exponent 0)
    // and 1.5 to 1.7 where every tile has value rows of 13 sizes from 2^-12 to 1.
    auto share = [&](auto role) {
        role(std::false_type(), r_all);
        if constexpr (Q8) {
            qt_fence_before();
            __syncthreads();
            if (*abort_flag != CK_BY_KEY) return;
            const PgRun r = ck_run_behind(srun);
            __syncthreads();
            if (threadIdx.x == 0) *abort_flag = 0u;
            __syncthreads();
            qt_fence_after();
            role(std::true_type(), r);
        }
    };

    if (warp >= 8 && warp < 12) {
    ck_reg_dec<C::R_CTL>();
    if (warp == 8) {
        // ------------------------------------------------ copies (TMA)
        share([&](auto pass, PgRun r) {
        constexpr bool BY_KEY = decltype(pass)::value;
        const CkBars<Q8> bar(bars + (BY_KEY ? C::BARS : 0));
        const int box = min(1 << p.c.page_shift, PG_TILE), nbox = PG_TILE / box;
        const int rows_all = p.c.num_pages * p.c.Hkv << p.c.page_shift;  // no box holds this row: reads zeros
        const uint64_t pol = ck_policy();
        [[maybe_unused]] PgRing<STAGES> kv;
        [[maybe_unused]] PgRing<C::RAW ? C::RAW : 1> raw;
        uint32_t qpar = 0;
        int tiles = 0, queries = 0;  // copied
        bool ok = true;
        do {
            if (queries > 0) {
                ok = __all_sync(FULL_MASK, wait(bar.q_empty, qpar));
                qpar ^= 1u;
                if (!ok) break;
            }
            ++queries;
            if (elect_lane()) {
                // tokens past the chunk bring other sequences' rows, past the tensor zeros: never used
                const int nq = r.e.nt > tqt ? 2 : 1;
                mbar_arrive_expect_tx(bar.q_full, (uint32_t)(nq * 2 * tqt * p.GQ * 128));
                for (int w = 0; w < nq; ++w)
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_3d(sq + w * TILE_B + hf * HALF_B, &p.tmq, 64 * hf, r.h * p.GQ, r.e.tok0 + w * tqt, bar.q_full, pol);
            }
            PgView view;
            view.set(r.e, p.window, p.sinks);
            int row = rows_all, prow = rows_all;  // of this tile and of the one before
            bool held = false;
            // in the order of use: keys of tile t + 1, then values of tile t
            for (int t = r.t0; t <= r.tn && ok; ++t) {
                prow = row;
                row = rows_all;
                held = false;
                if (t < r.tn) {
                    const int k0 = pg_tile_key(r.e, t) + lane * box;
                    if (lane < nbox && view.any(k0, k0 + box)) {
                        const int lp = k0 >> p.c.page_shift;
                        const int page = lp < p.max_pages ? __ldg(p.table + (long long)r.e.b * p.max_pages + lp) : -1;
                        held = page >= 0 && page < p.c.num_pages;
                        if (held) row = ((page * p.c.Hkv + r.h) << p.c.page_shift) + (k0 & ((1 << p.c.page_shift) - 1));
                        else atomicOr(&g_pk_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
                    }
                }
                if (Q8 && !BY_KEY && *abort_flag) {  // (the others then wait in vain, and stop)
                    ok = false;
                    break;
                }
                for (int part = 0; part < 2; ++part) {  // keys, values
                    if (part == 0 ? t == r.tn : t == r.t0) continue;
                    const CUtensorMap *map = part ? &p.tmv : &p.tmk;
                    const int at = part ? prow : row;
                    if constexpr (Q8) {
                        if (tiles >= C::RAW && !__all_sync(FULL_MASK, wait(&bar.raw_empty[raw.s], raw.par ^ 1u))) {
                            ok = false;
                            break;
                        }
                        // a key tile brings the exponents of keys and values
                        const unsigned n = part ? 0u : (unsigned)__popc(__ballot_sync(FULL_MASK, held));
                        if (BY_KEY && part == 0 && lane < nbox) srow[raw.s * 8 + lane] = held ? row : -1;
                        __syncwarp();
                        if (elect_lane()) mbar_arrive_expect_tx(&bar.raw_full[raw.s], RAW_B + n * 2 * box);
                        __syncwarp();
                        if (lane < nbox) {  // a lane per box
                            tma_load_2d(sraw + raw.s * RAW_B + lane * box * 128, map, 0, at, &bar.raw_full[raw.s], pol);
                            if (held && part == 0) {
                                unsigned char *x = sexp + raw.s * 2 * PG_TILE + lane * box;
                                bulk_g2s(x, p.c.ke + at, box, &bar.raw_full[raw.s], pol);
                                bulk_g2s(x + PG_TILE, p.c.ve + at, box, &bar.raw_full[raw.s], pol);
                            }
                        }
                        __syncwarp();
                        raw.step();
                    } else {
                        if (tiles >= STAGES && !__all_sync(FULL_MASK, wait(&bar.kv_empty[kv.s], kv.par ^ 1u))) {
                            ok = false;
                            break;
                        }
                        if (elect_lane()) mbar_arrive_expect_tx(&bar.kv_full[kv.s], TILE_B);
                        __syncwarp();
                        if (lane < nbox) {  // a lane per box
                            unsigned char *dst = skv + kv.s * TILE_B + lane * box * 128;
                            tma_load_2d(dst, map, 0, at, &bar.kv_full[kv.s], pol);
                            tma_load_2d(dst + HALF_B, map, 64, at, &bar.kv_full[kv.s], pol);
                        }
                        __syncwarp();
                        kv.step();
                    }
                    ++tiles;
                }
            }
        } while (ok && r.next(p.large, p.Hkv));
        // every copy has landed before the CTA may exit, or goes through its share
        // again (the last queries' too: nobody may have waited for them)
        if (queries > 0) (void)mbar_wait_bounded(bar.q_full, (uint32_t)(queries - 1) & 1u);
        if constexpr (Q8) {
            for (int k = 0; k < C::RAW && k < tiles; ++k) {
                const int j = tiles - 1 - k;
                (void)mbar_wait_bounded(&bar.raw_full[j % C::RAW], (uint32_t)(j / C::RAW) & 1u);
            }
        } else {
            for (int k = 0; k < STAGES && k < tiles; ++k) {
                const int j = tiles - 1 - k;
                (void)mbar_wait_bounded(&bar.kv_full[j % STAGES], (uint32_t)(j / STAGES) & 1u);
            }
        }
        __syncwarp();
        });
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------ products: warp 9 the
        // scores, warp 10 the values, so that neither's waits hold the other up
        // (one warp for both spent 3600 cycles a tile on waits and issues alone)
        constexpr uint32_t ID_S = ck_idesc(BFV, false), ID_O = ck_idesc(BFV, true);
        const uint64_t dq = qt_desc(smem_u32(sq)), dk = qt_desc(smem_u32(skv)), dv = ck_desc_v(smem_u32(skv));
        const uint32_t tm = __shfl_sync(FULL_MASK, tmem, 0);
        share([&](auto pass, PgRun r) {
        constexpr bool BY_KEY = decltype(pass)::value;
        const CkBars<Q8> bar(bars + (BY_KEY ? C::BARS : 0));
        PgRing<STAGES> kv;
        bool ok = true;
        auto await = [&](uint64_t *bar, uint32_t parity) { ok = ok && __all_sync(FULL_MASK, wait(bar, parity)); };
        if (warp == 9) {
            uint32_t qpar = 0, fpar = 1;  // (the score tile is free at first)
            int tiles = 0;                // of the ring, keys and values
            do {
                const bool two = r.e.nt > tqt;
                // A run's first keys may follow values in their slot: those must
                // have come and gone, or their pass would be taken for this one
                // (a barrier's parity tells two passes apart, not three).  Later
                // keys follow keys, or (codes) come in order.
                if (!Q8 && tiles >= STAGES) await(&bar.kv_empty[kv.s], kv.par ^ 1u);
                tiles += 2 * (r.tn - r.t0);
                await(QC ? bar.q_ready : bar.q_full, qpar);
                qpar ^= 1u;
                for (int t = r.t0; t < r.tn && ok; ++t) {
                    await(&bar.kv_full[kv.s], kv.par);
                    for (int w = 0; w < (two ? 2 : 1); ++w) {
                        await(bar.s_free, fpar);  // the score tile's last use was copied out
                        fpar ^= 1u;
                        if (!ok) break;
                        qt_fence_after();
                        ck_mma_ss(tm, dq + w * (TILE_B >> 4), dk + kv.s * (TILE_B >> 4), ID_S, smem_u32(&bar.s_full[w]));
                    }
                    if (!ok) break;
                    ck_commit(&bar.kv_empty[kv.s]);
                    kv.step();
                    if (t > r.t0) kv.step();  // (values of tile t - 1 lie between)
                }
                if (!ok) break;
                ck_commit(bar.q_empty);  // the queries may be replaced
                kv.step();
            } while (r.next(p.large, p.Hkv));
        } else {
            uint32_t ppar[2] = {0, 0};
            do {
                const bool two = r.e.nt > tqt;
                kv.step();
                for (int t = r.t0; t < r.tn && ok; ++t) {
                    if (t + 1 < r.tn) kv.step();  // (keys of tile t + 1 come first)
                    await(&bar.kv_full[kv.s], kv.par);
                    for (int w = 0; w < (two ? 2 : 1); ++w) {
                        await(&bar.p_full[w], ppar[w]);
                        ppar[w] ^= 1u;
                        if (!ok) break;
                        qt_fence_after();
                        ck_mma_ts(tm + 256 + 128 * w, tm + 128 + 64 * w, dv + kv.s * (TILE_B >> 4), ID_O, t > r.t0 ? 1u : 0u,
                                  smem_u32(&bar.pv_done[w]));
                    }
                    if (!ok) break;
                    ck_commit(&bar.kv_empty[kv.s]);
                    kv.step();
                }
            } while (ok && r.next(p.large, p.Hkv));
        }
        // every product is done before shared and tensor memory are given up
        ck_commit(&bar.drain[warp - 9]);
        (void)mbar_wait_bounded(&bar.drain[warp - 9], 0u);
        __syncwarp();
        });
    } else {
        share([](auto, PgRun) {});  // (takes part in the barriers)
    }
    } else if (warp < 8) {
        ck_reg_inc<C::R_SOFT>();
        // ------------------------------------------------ softmax: a thread per query row
        const int w = warp >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes, tp = tmem + lanes + 128 + 64 * w, to = tmem + lanes + 256 + 128 * w;
        const int tok_in = row / p.GQ;
        const float qabs = fabsf(p.qscale);
        const uint32_t keep = smem_u32(srun + 64 * warp);
        share([&](auto pass, PgRun r_) {
        constexpr bool BY_KEY = decltype(pass)::value;
        const CkBars<Q8> bar(bars + (BY_KEY ? C::BARS : 0));
        uint32_t spar = 0, vpar = 0, qpar = 0;
        PgRing<STAGES> vs;  // (16-bit cache) slot of the next tile that the products take
        PgRing<C::META ? C::META : 1> mt;
        bool ok = true;
        float back_q = 1.0f;  // undoes the power of two in this row of converted queries
        bool live = !QC;      // false: before the first item, whose queries are then made ready
        bool more = true;
        ck_keep(keep, r_, lane);
        do {
            const PgRun r = ck_run(keep);
            const bool rows = live && (w == 0 || r.e.nt > tqt);  // this half has rows in the item
            if (Q8 && live && !rows) {
                for (int t = r.t0; t < r.tn && ok; ++t) {
                    ok = __all_sync(FULL_MASK, wait(&bar.meta_full[mt.s], mt.par));  // (not ahead of its tile)
                    if (lane == 0) mbar_arrive(&bar.meta_empty[mt.s]);
                    mt.step();
                }
                if (!ok) break;
            }
            PgView view;
            view.set(r.e, p.window, p.sinks);
            const int tok = w * tqt + tok_in;
            const bool mine = tok_in < tqt && tok < r.e.nt;
            const int pos = mine ? r.e.p0 + tok : -1;
            const int low = p.window > 0 ? pos - p.window + 1 : 0;
            const int pos_a = r.e.p0 + w * tqt, pos_z = r.e.p0 + min(r.e.nt, (w + 1) * tqt) - 1;  // this tile's tokens
            float m = NEG_INF, l = 0.0f;
            if (rows) vs.step();
            for (int t = rows ? r.t0 : r.tn; t < r.tn; ++t) {
                const int k0 = pg_tile_key(r.e, t);
                if (t + 1 < r.tn) vs.step();  // now at the values of tile t
                const bool whole = k0 + PG_TILE <= pos_a + 1 &&
                                   (p.window == 0 || k0 > pos_z - p.window || k0 + PG_TILE <= view.sink);
                ok = __all_sync(FULL_MASK, wait(&bar.s_full[w], spar));
                spar ^= 1u;
                if (!ok) break;
                if constexpr (Q8) {
                    ok = __all_sync(FULL_MASK, wait(&bar.meta_full[mt.s], mt.par));
                    if (!ok) break;
                }
                qt_fence_after();
                // all scores of the row into registers
                uint32_t x[4][32];
#pragma unroll
                for (int b = 0; b < 4; ++b) qt_ld32(ts + 32 * b, x[b]);
                qt_wait_ld();
#pragma unroll
                for (int b = 0; b < 4; ++b) qt_hold(x[b]);
                qt_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.s_free);
                // t = score * mul + add, in base 2
                float mul = qabs, add = 0.0f, back = 1.0f;
                bool own = false;  // the keys' own exponents
                if constexpr (Q8) {
                    const float4 f = smeta[mt.s];
                    mul = QC ? fminf(fmaxf(f.x * back_q, 1e-37f), 3e38f) : f.x;  // (finite, and -inf times it stays)
                    add = f.y;
                    back = f.z;
                    if constexpr (BY_KEY) own = f.w != 0.0f;
                    if (!own) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.meta_empty[mt.s]);
                        mt.step();
                    }
                }
                if (p.qscale < 0.0f) {  // (mul is |scale|)
#pragma unroll
                    for (int c = 0; c < PG_TILE; ++c) x[c >> 5][c & 31] ^= 0x80000000u;
                }
                if (BY_KEY && own) {
                    const float4 *k2 = skeys + mt.s * (PG_TILE / 2);
#pragma unroll
                    for (int c = 0; c < PG_TILE; c += 2) {
                        const float4 f = k2[c >> 1];
                        uint32_t &a = x[c >> 5][c & 31], &b = x[c >> 5][(c & 31) + 1];
                        a = __float_as_uint(fmaf(__uint_as_float(a), QC ? fminf(f.x * back_q, 3e38f) : f.x, f.y));
                        b = __float_as_uint(fmaf(__uint_as_float(b), QC ? fminf(f.z * back_q, 3e38f) : f.z, f.w));
                    }
                    mul = 1.0f;
                    add = 0.0f;
                }
                if (!whole) {
                    // bit c of word b: key k0 + 32 b + c is seen (words, not
                    // comparisons key by key: those became branches)
                    const int hi = pos - k0 + 1, lo = low - k0, sink = view.sink - k0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t see = ck_below(hi - 32 * b) & (~ck_below(lo - 32 * b) | ck_below(sink - 32 * b));
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[b][j] = (see >> j) & 1u ? x[b][j] : 0xff800000u;
                    }
                }
                float mx4[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) mx4[b] = fmaxf(__uint_as_float(x[b][0]), __uint_as_float(x[b][1]));
#pragma unroll
                for (int j = 2; j < 32; j += 2)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        mx4[b] = fmaxf(fmaxf(mx4[b], __uint_as_float(x[b][j])), __uint_as_float(x[b][j + 1]));
                float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                mx = Q8 ? fmaf(mx, mul, add) : mx * mul;
                const bool grow = mx - OFF > m + LAG;
                bool used = t == r.t0;  // the last weights are used up, the output holds their product
                if (__any_sync(FULL_MASK, grow)) {
                    const float f = grow ? ex2(m - (mx - OFF)) : 1.0f;
                    if (grow) m = mx - OFF;
                    l *= f;
                    if (!used) {
                        ok = __all_sync(FULL_MASK, wait(&bar.pv_done[w], vpar));
                        vpar ^= 1u;
                        if (!ok) break;
                        used = true;
                        qt_fence_after();
#pragma unroll 1
                        for (int b = 0; b < 8; ++b) {
                            uint32_t y[16];
                            ck_ld16(to + 16 * b, y);
                            qt_wait_ld();
                            ck_hold16(y);
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                            ck_st16(to + 16 * b, y);
                        }
                    }
                }
                const float ms = m > NEG_INF ? m : 0.0f;
                if (BY_KEY && own) {  // sum w_j 2^-b_j
                    const float4 *k2 = skeys + mt.s * (PG_TILE / 2);
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int c = 0; c < PG_TILE; c += 2) {
                        const float4 f = k2[c >> 1];
                        s0 += ex2(__uint_as_float(x[c >> 5][c & 31]) - f.y - ms);
                        s1 += ex2(__uint_as_float(x[c >> 5][(c & 31) + 1]) - f.w - ms);
                    }
                    l += s0 + s1;
                    back = 0.0f;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.meta_empty[mt.s]);
                    mt.step();
                }
                const float2 neg = make_float2(add - ms, add - ms), mul2 = make_float2(mul, mul);
                float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 u = __ffma2_rn(ck_f2(x[b][j], x[b][j + 1]), mul2, neg);
                        const float2 e = make_float2(ex2(u.x), ex2(u.y));
                        sum2 = __fadd2_rn(sum2, e);
                        pk[j >> 1] = ck_pack<TV>(e.x, e.y);
                    }
                    if (b == 0 && !used) {
                        ok = __all_sync(FULL_MASK, wait(&bar.pv_done[w], vpar));
                        vpar ^= 1u;
                        if (!ok) break;
                        qt_fence_after();
                    }
                    ck_st16(tp + 16 * b, pk);
                }
                if (!ok) break;
                l = fmaf(sum2.x + sum2.y, back, l);
                if constexpr (!Q8) {
                    // values of keys that no row sees may hold anything: zero
                    // them before the product (the second half's comes later)
                    if (w == 0 && (k0 + PG_TILE > view.hi || (k0 < view.lo && k0 + PG_TILE > view.sink))) {
                        ok = __all_sync(FULL_MASK, wait(&bar.kv_full[vs.s], vs.par));
                        if (!ok) break;
                        if (!view.one(k0 + row)) {
                            uint4 *z = reinterpret_cast<uint4 *>(skv + vs.s * TILE_B + row * 128);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                z[j] = make_uint4(0u, 0u, 0u, 0u);
                                z[HALF_B / 16 + j] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        fence_proxy_async_smem();
                    }
                }
                vs.step();
                ck_wait_st();
                qt_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[w]);
            }
            if (!ok) break;
            if (rows) {
                ok = __all_sync(FULL_MASK, wait(&bar.pv_done[w], vpar));
                vpar ^= 1u;
                if (!ok) break;
                qt_fence_after();
            }
            PgRun z = ck_run(keep);
            if (QC && (!live || z.left > z.tn - z.t0)) {
                // the next item's queries, before the output of this one (both
                // halves, whether they will have rows or not: what a tile without
                // rows holds is not used)
                ok = __all_sync(FULL_MASK, wait(bar.q_full, qpar));
                qpar ^= 1u;
                if (!ok) break;
                back_q = ck_query(sq + w * TILE_B, row);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.q_ready);
            }
            if (live && (w == 0 || z.e.nt > tqt)) {
                const int tok = w * tqt + tok_in;
                const bool mine = tok_in < tqt && tok < z.e.nt;
                const bool split = z.t0 > 0 || z.tn < z.e.ntiles;
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                float *part = p.large.part + (size_t)(2 * blockIdx.x + (z.first && z.t0 > 0 ? 0 : 1)) * (PG_LROWS * PG_PART);
                if (split && mine) {
                    part[128 * w + row] = m;
                    part[PG_LROWS + 128 * w + row] = l;
                }
                // A thread holds a row and stores 32 bytes of it at a time, a whole
                // sector.  Partial rows lie 32 by 32, 8 columns after another, so that a
                // warp's store fills whole lines (row after row, a sector of a line
                // each, an item's output took 2.1 us, so 1.3).
                T *dst = static_cast<T *>(p.out) + ((size_t)(z.e.tok0 + tok) * p.Hq + (size_t)z.h * p.GQ + row % p.GQ) * D;
                float *pd = part + 2 * PG_LROWS + (128 * w + row - lane) * D + 8 * lane;
                const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t y[32];
                    qt_ld32(to + 32 * b, y);
                    qt_wait_ld();
                    qt_hold(y);
                    if (mine && split) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ck_store32(pd + 256 * (4 * b + i), y + 8 * i);
                    } else if (mine) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t v[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                v[c] = ck_pack<T>(__uint_as_float(y[16 * i + 2 * c]) * inv, __uint_as_float(y[16 * i + 2 * c + 1]) * inv);
                            if (wide) {
                                ck_store32(dst + 32 * b + 16 * i, v);
                            } else {
                                uint4 *to16 = reinterpret_cast<uint4 *>(dst + 32 * b + 16 * i);
                                to16[0] = make_uint4(v[0], v[1], v[2], v[3]);
                                to16[1] = make_uint4(v[4], v[5], v[6], v[7]);
                            }
                        }
                    }
                    __syncwarp();
                }
                qt_fence_before();  // (ordered before the next run's products by bar.p_full)
            }
            if (live) {
                more = z.next(p.large, p.Hkv);
                ck_keep(keep, z, lane);
            }
            live = true;
        } while (more);
        });
    } else if constexpr (Q8) {
        ck_reg_dec<C::R_CONV>();
        // ------------------------------------------------ codes to 16-bit operands
        const int j = threadIdx.x - 12 * 32;
        constexpr int STEP = 4 * C::CONV, ROWS = PG_TILE / STEP;
        static_assert(ROWS == 4, "a byte each of a word");
        share([&](auto pass, PgRun r) {
        constexpr bool BY_KEY = decltype(pass)::value;
        const CkBars<Q8> bar(bars + (BY_KEY ? C::BARS : 0));
        PgRing<C::RAW ? C::RAW : 1> raw;
        PgRing<STAGES> kv;
        PgRing<C::META ? C::META : 1> mt;
        int tiles = 0, keys = 0;
        const int box = min(1 << p.c.page_shift, PG_TILE);
        uint32_t far = 0u;  // exponents of this lane's keys too far below the tile's largest
        int vtop0 = 0, vtop1 = 0;  // exponents of the values to come: of tile u - 1, of tile u
        uint32_t vrow0 = 0, vrow1 = 0;
        bool ok = true;
        do {
            PgView view;
            view.set(r.e, p.window, p.sinks);
            for (int u = r.t0; u <= r.tn && ok; ++u) {
                for (int part = 0; part < 2; ++part) {  // keys of tile u, values of the tile before
                    if (part == 0 ? u == r.tn : u == r.t0) continue;
                    const int k0 = pg_tile_key(r.e, part ? u - 1 : u);
                    const bool edge = k0 + PG_TILE > view.hi || (k0 < view.lo && k0 + PG_TILE > view.sink);
                    ok = __all_sync(FULL_MASK, wait(&bar.raw_full[raw.s], raw.par));
                    if (ok && tiles >= STAGES) ok = __all_sync(FULL_MASK, wait(&bar.kv_empty[kv.s], kv.par ^ 1u));
                    if (ok && part == 0 && keys >= C::META) ok = __all_sync(FULL_MASK, wait(&bar.meta_empty[mt.s], mt.par ^ 1u));
                    if (!ok) break;
                    // rows of this thread: j / 8 + 4 CONV i
                    int top;              // the tile's largest exponent; 0: codes are taken as they are
                    uint32_t rows = 0;    // this thread's rows' exponents, a byte each
                    if (part == 0) {
                        const uint32_t *e4 = reinterpret_cast<const uint32_t *>(sexp + raw.s * 2 * PG_TILE) + lane;
                        const uint32_t ke = e4[0];
                        uint32_t ve = e4[PG_TILE / 4];
                        uint32_t see = 0xffffffffu;  // of this lane's four keys
                        if (edge) {
                            see = 0u;
#pragma unroll
                            for (int i = 0; i < 4; ++i) see |= view.one(k0 + 4 * lane + i) ? 0xffu << (8 * i) : 0u;
                        }
                        top = ck_top(ke & see);
                        vtop1 = ck_top(ve & see);
                        if constexpr (BY_KEY) {
                            if (vtop1 >= 127) {
                                const uint32_t exp0 = __vcmpeq4(ve | ~see, PG_EXP0);
                                const int rw = exp0 != 0u ? srow[raw.s * 8 + 4 * lane / box] : -1;
                                if (rw >= 0)
                                    ve = pg_value_exps(ve | ~see, static_cast<const unsigned char *>(p.c.v) + (long long)(rw + 4 * lane % box) * D);
                                vtop1 = ck_top(ve & see);
                            }
                        }
                        far = ck_less(ke | ~see, top - KEYS_WITHIN) | ck_less(ve | ~see, vtop1 - VALUES_WITHIN);
                        top = max(top, 87);  // (at least 2^-40: the factors below stay normal)
                        vtop1 = max(vtop1, 87);
                        const unsigned char *ex = sexp + raw.s * 2 * PG_TILE + (j >> 3);
                        vrow1 = 0;
#pragma unroll
                        for (int i = ROWS - 1; i >= 0; --i) {
                            rows = rows << 8 | ex[STEP * i];
                            vrow1 = vrow1 << 8 | ex[PG_TILE + STEP * i];
                        }
                        const bool own = BY_KEY && __any_sync(FULL_MASK, far != 0u);  // the keys' own exponents
                        if (j == 0) {
                            const int A = top - 127, B = vtop1 - 127;
                            // (the factor stays a number that -inf times it stays -inf, however small the scale)
                            smeta[mt.s] = make_float4(fmaxf(fabsf(p.qscale) * pow2f(min(A, 127)), 1e-37f), (float)B,
                                                      pow2f(max(-B, -126)), own ? 1.0f : 0.0f);
                        }
                        if (own) {  // each warp writes an even share of the keys, four a lane
                            if (lane / (32 / C::CONV) == (j >> 5)) {
#pragma unroll 1
                                for (int i = 0; i < 2; ++i) {
                                    const int a = (int)(ke >> (16 * i)), b = (int)(ve >> (16 * i));
                                    auto f = [&](int e) { return fabsf(p.qscale) * pow2f(min(max((e & 0xff) - 127, -126), 127)); };
                                    skeys[mt.s * (PG_TILE / 2) + 2 * lane + i] =
                                        make_float4(f(a), (float)((b & 0xff) - 127), f(a >> 8), (float)(((b >> 8) & 0xff) - 127));
                                }
                            }
                            top = vtop1 = 0;
                        }
                    } else {
                        top = vtop0;
                        rows = vrow0;
                    }
                    // (a short loop: unrolled in full, the warps' code no longer
                    // fitted the instruction caches and a chunk took twice as long)
                    const unsigned char *src = sraw + raw.s * RAW_B + swz128(j >> 3, j & 7);  // 16 rows on: the same swizzle
                    unsigned char *dst = skv + kv.s * TILE_B + ((j & 7) >> 2) * HALF_B;
                    // eight lanes hold a row; the upper four store their second half
                    // first, so that the eight fill all banks
                    const bool odd = (j & 4) != 0;
                    const uint32_t d0 = swz128(j >> 3, 2 * (j & 3) + odd), d1 = swz128(j >> 3, 2 * (j & 3) + !odd);
                    const bool hide = edge && part == 1;  // values of keys that no row sees may hold anything
#pragma unroll 2
                    for (int i = 0; i < ROWS; ++i, rows >>= 8) {
                        uint4 v = *reinterpret_cast<const uint4 *>(src + 128 * STEP * i);
                        if (hide && !view.one(k0 + (j >> 3) + STEP * i)) v = make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t f = ck_factor((int)(rows & 0xffu) - top);
                        uint4 x0, x1;
                        ck_operand(odd ? v.z : v.x, f, x0.x, x0.y);
                        ck_operand(odd ? v.w : v.y, f, x0.z, x0.w);
                        ck_operand(odd ? v.x : v.z, f, x1.x, x1.y);
                        ck_operand(odd ? v.y : v.w, f, x1.z, x1.w);
                        *reinterpret_cast<uint4 *>(dst + d0 + 128 * STEP * i) = x0;
                        *reinterpret_cast<uint4 *>(dst + d1 + 128 * STEP * i) = x1;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.raw_empty[raw.s]);
                        mbar_arrive(&bar.kv_full[kv.s]);
                        if (part == 0) mbar_arrive(&bar.meta_full[mt.s]);
                    }
                    raw.step();
                    kv.step();
                    ++tiles;
                    if (part == 0) {
                        mt.step();
                        ++keys;
                        // (exponent 0, or more: there may be zero rows)
                        if (!BY_KEY && (__any_sync(FULL_MASK, far != 0u) || vtop1 >= 127)) {
                            *abort_flag = CK_BY_KEY;
                            ok = false;
                            break;
                        }
                    }
                }
                vtop0 = vtop1;
                vrow0 = vrow1;
            }
        } while (ok && r.next(p.large, p.Hkv));
        });
    }

    qt_fence_before();
    __syncthreads();
    qt_fence_after();
    if (warp == 9) tmem_free(tmem, 512);
}

template <class T, bool Q8>
cudaError_t launch_chunk(const PagedAttendParams &p, cudaStream_t stream)
{
    auto kern = paged_chunk_kernel<T, Q8>;
    constexpr int smem = CkShape<Q8>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // The warps trade registers inside the launch's share, and a warp that asks for
    // more than is there waits forever: never start with fewer than the shares add up
    // to.  (The compiler gives such a kernel what its launch bounds allow, which is
    // REGS.)
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return e;
        regs.store(at.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < CkShape<Q8>::REGS) return cudaErrorLaunchOutOfResources;
    return launch_early(kern, dim3(p.large.G), CkShape<Q8>::THREADS, smem, stream, p);
}

}  // namespace

cudaError_t launch_paged_large(const PagedAttendParams &p0, int q_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAttendParams p = p0;
    const bool q8 = cache_dtype == VQ_E4M3;
    const uint64_t rows = ((uint64_t)p.c.num_pages * p.c.Hkv) << p.c.page_shift;
    const uint32_t box = 1u << p.c.page_shift < (unsigned)PG_TILE ? 1u << p.c.page_shift : (unsigned)PG_TILE;
    if (!encode_tmap_pages(&p.tmk, p.c.k, rows, q8 ? 1 : 2, box) || !encode_tmap_pages(&p.tmv, p.c.v, rows, q8 ? 1 : 2, box))
        return cudaErrorInvalidValue;
    // queries: boxes of 64 columns, the heads of a kv head, the tokens of a tile
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.Hq, (uint64_t)p.T};
    const uint64_t strides[2] = {(uint64_t)(p.Hq > 1 ? p.qsh : D) * 2, (uint64_t)(p.T > 1 ? p.qst : (long long)p.Hq * D) * 2};
    const uint32_t qbox[3] = {64u, (uint32_t)p.GQ, (uint32_t)(128 / p.GQ)};
    if (!encode_tmap_f16(&p.tmq, p.q, 3, dims, strides, qbox, true, true)) return cudaErrorInvalidValue;
    if (q_dtype == VQ_F16) return q8 ? launch_chunk<__half, true>(p, stream) : launch_chunk<__half, false>(p, stream);
    return q8 ? launch_chunk<__nv_bfloat16, true>(p, stream) : launch_chunk<__nv_bfloat16, false>(p, stream);
}

cudaError_t paged_chunk_take_device_error(unsigned *bits, cudaStream_t stream)
{
    *bits = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_pk_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (*bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_pk_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace vq
