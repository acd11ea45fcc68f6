// paged_attend.cu - attention of new tokens over a paged key/value cache
// (sm_103a): the plan that shares the work out, the kernel for few query rows
// per kv head (single tokens and short continuations), and the merge of
// partial results.
//
// For the new token i of sequence b at position p = lens[b] - n_b + i,
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j - max),
// over the keys j <= p with (no window, or j > p - window, or j < sinks).  Rows
// that see no key give zeros.
//
// 8-bit cache.  With k_j = 2^a_j K_j and v_j = 2^b_j V_j (codes K, V exact in
// fp16 and bf16) the score is 2^a_j (q . K_j), and the exponent of the value is
// folded into the weight: w'_j = 2^(s_j + b_j - M) with M the maximum of
// s_j + b_j, so that w' is at most 1 whatever the exponents, out = sum w'_j V_j
// / sum w'_j 2^-b_j, and the products take codes that were never scaled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pa_err);

constexpr int D = 128;
constexpr float NEG_INF = -__builtin_huge_valf();

// ---------------------------------------------------------------- the plan

constexpr int PLAN_THREADS = 1024;

// Exclusive sum over the block; `total` gets the sum of all.
__device__ __forceinline__ long long block_scan(long long v, long long *ws, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, x, s);
        if (lane >= s) x += y;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long y = ws[lane];
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const long long z = __shfl_up_sync(FULL_MASK, y, s);
            if (lane >= s) y += z;
        }
        ws[lane] = y;
    }
    __syncthreads();
    const long long before = warp ? ws[warp - 1] : 0;
    total = ws[31];
    __syncthreads();
    return before + x - v;
}

__device__ __forceinline__ PgEntry make_entry(const PagedAttendParams &p, int b, int start, int n, int len, int tq, int i)
{
    PgEntry e;
    e.b = b;
    e.tok0 = start + i * tq;
    e.nt = min(tq, n - i * tq);
    e.p0 = len - n + i * tq;
    e.hi = max(0, e.p0 + e.nt);
    const int lo = p.window > 0 ? max(0, e.p0 - p.window + 1) : 0;
    const int sink = p.window > 0 ? min(p.sinks, e.hi) : 0;
    const int th = (e.hi + PG_TILE - 1) / PG_TILE, st = (sink + PG_TILE - 1) / PG_TILE, tl = lo / PG_TILE;
    // leading tiles that reach the window make one run with it
    e.nsink = st >= tl ? 0 : st;
    e.tl = st >= tl ? 0 : tl;
    e.ntiles = max(1, e.nsink + th - e.tl);
    return e;
}

// One CTA: entries of both classes in the order of the sequences, the units
// before each, and where each CTA of the attention kernels starts.
__global__ void __launch_bounds__(PLAN_THREADS, 1) paged_plan_kernel(const __grid_constant__ PagedAttendParams p)
{
    __shared__ long long ws[32];
    const int lane = threadIdx.x & 31;
    const int cap_len = (int)min((long long)p.max_pages << p.c.page_shift, 0x7fffffffLL);
    long long carry = 0;  // entries so far: small in the low half, large in the high one
    for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        int start = 0, n = 0, len = 0;
        if (b < p.B) {
            start = min(max(p.cu[b], 0), p.T);
            n = min(max(p.cu[b + 1], start), p.T) - start;
            len = min(max(p.lens[b], 0), cap_len);
            if (n > p.max_q) {
                atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
                n = p.max_q;
            }
        }
        const bool large = n * p.GQ > p.small_rows;
        const int tq = large ? p.large.tq : p.small.tq;
        const int cnt = (n + tq - 1) / tq;
        long long all;
        const long long off = carry + block_scan(large ? (long long)cnt << 32 : cnt, ws, all);
        carry += all;
        const int first = (int)(large ? off >> 32 : off & 0xffffffffLL);
        // sequences of one entry write it themselves, a warp writes those of more
        auto put = [&](int b_, int start_, int n_, int len_, bool large_, int first_, int i) {
            const PgPlan &pl = large_ ? p.large : p.small;
            if (first_ + i < pl.cap) pl.ent[first_ + i] = make_entry(p, b_, start_, n_, len_, pl.tq, i);
            else atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        };
        if (cnt == 1) put(b, start, n, len, large, first, 0);
        unsigned many = __ballot_sync(FULL_MASK, cnt > 1);
        while (many) {
            const int l = __ffs(many) - 1;
            many &= many - 1;
            const int b_ = __shfl_sync(FULL_MASK, b, l), s_ = __shfl_sync(FULL_MASK, start, l);
            const int n_ = __shfl_sync(FULL_MASK, n, l), len_ = __shfl_sync(FULL_MASK, len, l);
            const int f_ = __shfl_sync(FULL_MASK, first, l), c_ = __shfl_sync(FULL_MASK, cnt, l);
            const bool g_ = __shfl_sync(FULL_MASK, (int)large, l) != 0;
            for (int i = lane; i < c_; i += 32) put(b_, s_, n_, len_, g_, f_, i);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const PgPlan &pl = k ? p.large : p.small;
        if (pl.cap == 0) continue;
        const int nent = min(pl.cap, (int)(k ? carry >> 32 : carry & 0xffffffffLL));
        long long total = 0;
        for (int i0 = 0; i0 < nent; i0 += PLAN_THREADS) {
            const int i = i0 + threadIdx.x;
            const long long u = i < nent ? (long long)pl.ent[i].ntiles * p.Hkv : 0;
            long long all;
            const long long before = block_scan(u, ws, all);
            if (i < nent) pl.base[i] = total + before;
            total += all;
        }
        __syncthreads();
        PgPlanHead h;
        h.total = total;
        h.nent = nent;
        h.g = (int)min((long long)pl.G, total);
        if (threadIdx.x == 0) *pl.head = h;
        for (int c = threadIdx.x; c < h.g; c += PLAN_THREADS) {
            const long long u = pg_first_unit(h, c);
            int a = 0, z = nent - 1;  // the last entry that starts at or before u
            while (a < z) {
                const int m = (a + z + 1) >> 1;
                if (pl.base[m] <= u) a = m;
                else z = m - 1;
            }
            const int r = (int)(u - pl.base[a]), nt = pl.ent[a].ntiles;
            pl.ctab[c] = make_int4(a, r / nt, r % nt, 0);
        }
    }
}

// ------------------------------------------------------- the merge of parts

constexpr int CB_ROWS = 16;  // rows of one combine CTA

template <class T> __device__ __forceinline__ uint2 pack4(float4 v);
template <> __device__ __forceinline__ uint2 pack4<__half>(float4 v)
{
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
template <> __device__ __forceinline__ uint2 pack4<__nv_bfloat16>(float4 v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// CTA c merges the item that c enters in its middle, if no earlier CTA does
// so: its parts are the second slot of CTA c - 1 and the first slots of c,
// c + 1, ..., in that order on every run.
template <class T, int ROWS, int HALF>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ PagedAttendParams p)
{
    const PgPlan &pl = HALF ? p.large : p.small;
    const PgPlanHead h = *pl.head;
    const int c = blockIdx.x;
    if (c == 0 || c >= h.g) return;
    const int4 at = pl.ctab[c];
    const long long u = pg_first_unit(h, c);
    if (at.z == 0 || at.z > u - pg_first_unit(h, c - 1)) return;
    const PgEntry e = pl.ent[at.x];
    const long long end = u - at.z + e.ntiles;
    int parts = 2;
    while (c + parts - 1 < h.g && pg_first_unit(h, c + parts - 1) < end) ++parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int RT = HALF ? 128 : ROWS;  // rows of one tile of queries
    const int tqt = RT / p.GQ;
    const size_t slot = (size_t)ROWS * PG_PART;
    for (int i = warp; i < CB_ROWS; i += 4) {
        const int r = blockIdx.y * CB_ROWS + i;
        const int tok = (r / RT) * tqt + (r % RT) / p.GQ, g = (r % RT) % p.GQ;
        if (r % RT >= tqt * p.GQ || tok >= e.nt) continue;
        float M = NEG_INF;
        for (int k = lane; k < parts; k += 32) {
            const float *s = pl.part + (size_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c + k - 1)) * slot;
            M = fmaxf(M, s[r]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
        float L = 0.0f;
        float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (M > NEG_INF) {
            for (int k = 0; k < parts; ++k) {
                const float *s = pl.part + (size_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c + k - 1)) * slot;
                const float f = ex2(s[r] - M);
                const float4 o = *reinterpret_cast<const float4 *>(s + 2 * ROWS + (size_t)r * D + 4 * lane);
                L = fmaf(s[ROWS + r], f, L);
                O.x = fmaf(o.x, f, O.x);
                O.y = fmaf(o.y, f, O.y);
                O.z = fmaf(o.z, f, O.z);
                O.w = fmaf(o.w, f, O.w);
            }
        }
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        O.x *= inv; O.y *= inv; O.z *= inv; O.w *= inv;
        T *dst = static_cast<T *>(p.out) + ((size_t)(e.tok0 + tok) * p.Hq + (size_t)at.y * p.GQ + g) * D + 4 * lane;
        *reinterpret_cast<uint2 *>(dst) = pack4<T>(O);
    }
}

// --------------------------------------------------------- the small kernel
//
// One CTA of 8 warps per SM.  A tile of 128 keys is cut into 16 keys for each
// warp; a warp streams its own 16-key blocks of keys and values by TMA through
// a ring of its own (no barrier between warps in the loop) and keeps the
// running maximum, sum and output of all 16 rows (new tokens x query heads of
// the kv head, so the cache is read once for all of them) in registers.  Both
// products are 16 x 8 x 16 mma.sync: HBM bounds this kernel, and a tile of 128
// tensor-memory rows would be mostly padding.  The order of the 128
// coordinates in the score product is free as long as both operands share it:
// each lane takes 16 consecutive bytes of its key's row per load, for fp16 and
// for codes alike.  The walk over the units continues across items, so the
// copies of the next item are in flight while an item's warps are merged.
constexpr int SM_WARPS = 8;
constexpr int KB = 16;  // keys of a warp's block
constexpr float OFF = 7.0f;    // weights reach up to 2^(OFF + LAG): fp16 stays normal down to 2^-14
constexpr float LAG = 8.0f;    // the maximum is only followed when it grew by more than this

constexpr int MROW = D + 4;    // row of the merge buffers (floats)

template <bool Q8> struct SmTile {
    static constexpr int ROW = Q8 ? 128 : 256;            // bytes of a cache row
    static constexpr int KV = KB * ROW;                   // keys, or values, of a block
    static constexpr int STAGE = 2 * KV;                  // keys, values
    static constexpr int STAGES = Q8 ? 5 : 3;
    static constexpr int EXP = Q8 ? 2 * KB : 0;           // exponents of a block
    static constexpr int MERGE = 4 * 16 * MROW * 4;       // four warps' outputs; maxima and sums in the padding
    static constexpr int SMEM = 1024 + SM_WARPS * STAGES * (STAGE + EXP + 8) + MERGE;
};
static_assert(SmTile<false>::SMEM <= 232448 && SmTile<true>::SMEM <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <class T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                     uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <class T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A pair of e4m3 codes as a pair of T (exact: both types hold every code).
template <class T> __device__ __forceinline__ uint32_t codes2(uint32_t two);
template <> __device__ __forceinline__ uint32_t codes2<__half>(uint32_t two) { return e4m3x2_to_f16x2(two); }
template <> __device__ __forceinline__ uint32_t codes2<__nv_bfloat16>(uint32_t two)
{
    const uint32_t h2 = e4m3x2_to_f16x2(two);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
    return pack2<__nv_bfloat16>(f.x, f.y);
}

// The walk of one warp over its CTA's units: the item (entry, head), the tile,
// and the units left.
struct Walk {
    PgEntry e;
    PgView v;
    int ei, h, t, left;
    __device__ __forceinline__ void load(const PagedAttendParams &p)
    {
        e = pg_entry(p.small.ent + ei);
        v.set(e, p.window, p.sinks);
    }
    __device__ __forceinline__ bool next(const PagedAttendParams &p)  // false: no unit left
    {
        if (--left <= 0) return false;
        if (++t == e.ntiles) {
            t = 0;
            if (++h == p.Hkv) {
                h = 0;
                ++ei;
                load(p);
            }
        }
        return true;
    }
};

// T: query and output type; Q8: e4m3 cache (values are then taken as fp16)
template <class T, bool Q8>
__global__ void __launch_bounds__(SM_WARPS * 32, 1) paged_small_kernel(const __grid_constant__ PagedAttendParams p)
{
    using L = SmTile<Q8>;
    using TV = typename std::conditional<Q8, __half, T>::type;  // operand type of the value product
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *stages = smem_1k(smem_raw);
    float *merge = reinterpret_cast<float *>(stages + SM_WARPS * L::STAGES * L::STAGE);
    unsigned char *exps = reinterpret_cast<unsigned char *>(merge + 4 * 16 * MROW);
    uint64_t *bars = reinterpret_cast<uint64_t *>(exps + SM_WARPS * L::STAGES * L::EXP);
    // maximum (and, one further, sum) of row r of warp w, in the padding of the merge buffers
    auto stat = [&](int w, int r) -> float * { return merge + ((w & 3) * 16 + r) * MROW + D + 2 * (w >> 2); };

    const PgPlanHead head = *p.small.head;
    const int c = blockIdx.x;
    if (c >= head.g) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    unsigned char *my_st = stages + warp * L::STAGES * L::STAGE;
    unsigned char *my_exp = exps + warp * L::STAGES * L::EXP;
    uint64_t *my_bar = bars + warp * L::STAGES;
    if (lane == 0) {
        for (int s = 0; s < L::STAGES; ++s) mbar_init(&my_bar[s], 1);
        fence_mbar_init();
    }
    __syncwarp();

    Walk co;  // what is computed
    {
        const int4 at = p.small.ctab[c];
        co.ei = at.x;
        co.h = at.y;
        co.t = at.z;
        co.left = (int)(pg_first_unit(head, c + 1) - pg_first_unit(head, c));
        co.load(p);
    }
    Walk is = co;  // what is copied
    bool more = true;
    int issued = 0, taken = 0;
    const uint64_t pol = l2_policy_evict_first();
    const int rows_all = p.c.num_pages * p.c.Hkv << p.c.page_shift;  // a row that no box holds: reads zeros
    auto issue = [&]() {  // the next block with a visible key, if any
        while (more) {
            const int k0 = pg_tile_key(is.e, is.t) + KB * warp;
            const bool see = is.v.any(k0, k0 + KB);
            if (see && lane == 0) {
                const int lp = k0 >> p.c.page_shift;
                int page = lp < p.max_pages ? __ldg(p.table + (long long)is.e.b * p.max_pages + lp) : -1;
                if (page < 0 || page >= p.c.num_pages) {
                    atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
                    page = -1;
                }
                const int row = page < 0 ? rows_all
                                         : ((page * p.c.Hkv + is.h) << p.c.page_shift) + (k0 & ((1 << p.c.page_shift) - 1));
                const int st = issued % L::STAGES;
                unsigned char *dst = my_st + st * L::STAGE;
                uint64_t *bar = &my_bar[st];
                if constexpr (Q8) {
                    mbar_arrive_expect_tx(bar, 2 * L::KV + (page < 0 ? 0 : 2 * KB));
                    tma_load_2d(dst, &p.tmk, 0, row, bar, pol);
                    tma_load_2d(dst + L::KV, &p.tmv, 0, row, bar, pol);
                    if (page >= 0) {
                        bulk_g2s(my_exp + st * L::EXP, p.c.ke + row, KB, bar, pol);
                        bulk_g2s(my_exp + st * L::EXP + KB, p.c.ve + row, KB, bar, pol);
                    }
                } else {
                    mbar_arrive_expect_tx(bar, 2 * L::KV);
                    tma_load_2d(dst, &p.tmk, 0, row, bar, pol);
                    tma_load_2d(dst + L::KV / 2, &p.tmk, 64, row, bar, pol);
                    tma_load_2d(dst + L::KV, &p.tmv, 0, row, bar, pol);
                    tma_load_2d(dst + L::KV + L::KV / 2, &p.tmv, 64, row, bar, pol);
                }
            }
            more = is.next(p);
            if (see) {
                ++issued;
                return;
            }
        }
    };
    for (int s = 0; s < L::STAGES; ++s) issue();

    bool ok = true, first_item = true;
    for (;;) {
        // ---- one item, or the part of it in this CTA's share
        const PgEntry e = co.e;
        const PgView v = co.v;
        const int h = co.h, t0 = co.t;
        const int tn = min(e.ntiles, t0 + co.left);
        const int rows = e.nt * p.GQ;
        // query fragments: lane's rows g8, g8 + 8; its run of coordinates per
        // 16 bytes of cache row (8 entries or 16 codes) at run t4 + 4 q
        constexpr int RUN = Q8 ? 16 : 8;
        uint32_t qf[2][16];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g8 + 8 * r;
            const bool in = row < rows;
            const T *src = static_cast<const T *>(p.q);
            if (in) src += (e.tok0 + row / p.GQ) * p.qst + ((long long)h * p.GQ + row % p.GQ) * p.qsh;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // the j-th 8 coordinates of this lane
                const int d = RUN == 8 ? 8 * (t4 + 4 * j) : 16 * (t4 + 4 * (j >> 1)) + 8 * (j & 1);
                const uint4 w = in ? __ldg(reinterpret_cast<const uint4 *>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
                qf[r][4 * j] = w.x;
                qf[r][4 * j + 1] = w.y;
                qf[r][4 * j + 2] = w.z;
                qf[r][4 * j + 3] = w.w;
            }
        }
        // visible keys of this lane's two rows: j <= pos, and the window
        int pos[2], low[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g8 + 8 * r;
            pos[r] = row < rows ? e.p0 + row / p.GQ : -1;
            low[r] = p.window > 0 ? pos[r] - p.window + 1 : 0;
        }
        const int lo_all = p.window > 0 ? e.p0 + e.nt - p.window : 0;  // the last row's first key in the window
        float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.0f, 0.0f};
        float o[16][4];
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.0f;

        for (int t = t0; t < tn; ++t) {
            const int k0 = pg_tile_key(e, t) + KB * warp;
            if (!v.any(k0, k0 + KB) || !ok) continue;
            const int st = taken % L::STAGES;
            if (!__all_sync(FULL_MASK, mbar_wait_bounded(&my_bar[st], (uint32_t)(taken / L::STAGES) & 1u))) {
                if (lane == 0) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
                ok = false;
                continue;
            }
            const unsigned char *sb = my_st + st * L::STAGE;
            // ---- scores: S[row][key], two blocks of 8 keys
            float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int key = 8 * nt + g8;
                if constexpr (Q8) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(sb + swz128(key, t4 + 4 * q));
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int i = 8 * q + 2 * j;  // pairs 2 i, 2 i + 1 of the lane's coordinates
                            mma16<T>(s[nt], qf[0][i], qf[1][i], qf[0][i + 1], qf[1][i + 1], codes2<T>(x[j] & 0xffffu),
                                     codes2<T>(x[j] >> 16));
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(sb + (q >> 1) * (L::KV / 2) +
                                                                         swz128(key, t4 + 4 * (q & 1)));
                        mma16<T>(s[nt], qf[0][4 * q], qf[1][4 * q], qf[0][4 * q + 1], qf[1][4 * q + 1], w.x, w.y);
                        mma16<T>(s[nt], qf[0][4 * q + 2], qf[1][4 * q + 2], qf[0][4 * q + 3], qf[1][4 * q + 3], w.z, w.w);
                    }
                }
            }
            // ---- scale, mask: this lane's keys are 8 nt + 2 t4 + {0, 1}
            float vb[2][2];  // 2^-b of the lane's keys' values (8-bit cache)
            const bool whole = k0 + KB <= e.p0 + 1 && (p.window == 0 || k0 >= lo_all || k0 + KB <= v.sink);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float a = p.qscale, b = 0.0f;
                    if constexpr (Q8) {
                        const int key = 8 * nt + 2 * t4 + j;
                        const int be = (int)my_exp[st * L::EXP + KB + key] - 127;
                        a *= pow2f(max((int)my_exp[st * L::EXP + key] - 127, -126));
                        b = (float)be;
                        vb[nt][j] = pow2f(max(-be, -126));
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float &x = s[nt][2 * r + j];
                        x = fmaf(x, a, b);
                        if (!whole) {
                            const int k = k0 + 8 * nt + 2 * t4 + j;
                            const bool in = k <= pos[r] && (k >= low[r] || k < v.sink);
                            x = in ? x : NEG_INF;
                        }
                    }
                }
            }
            // ---- softmax: the four lanes of a row share its maximum
            uint32_t pf[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, 1));
                x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, 2));
                if (x - OFF > m[r] + LAG) {  // the same for the row's four lanes
                    const float f = ex2(m[r] - (x - OFF));
                    m[r] = x - OFF;
                    l[r] *= f;
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        o[n][2 * r] *= f;
                        o[n][2 * r + 1] *= f;
                    }
                }
                const float mm = m[r] > NEG_INF ? m[r] : 0.0f;
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = ex2(s[i >> 1][2 * r + (i & 1)] - mm);
                if constexpr (Q8) {
                    l[r] += w[0] * vb[0][0] + w[1] * vb[0][1] + (w[2] * vb[1][0] + w[3] * vb[1][1]);
                } else {
                    l[r] += (w[0] + w[1]) + (w[2] + w[3]);
                }
                pf[r] = pack2<TV>(w[0], w[1]);
                pf[r + 2] = pack2<TV>(w[2], w[3]);
            }
            // ---- values: keys that no row sees may hold anything, their
            // entries are masked out of the operand
            uint32_t ka = 0xffffffffu, kb = 0xffffffffu;
            if (!whole) {
                const int k = k0 + 2 * t4;
                ka = (v.one(k) ? 0x0000ffffu : 0u) | (v.one(k + 1) ? 0xffff0000u : 0u);
                kb = (v.one(k + 8) ? 0x0000ffffu : 0u) | (v.one(k + 9) ? 0xffff0000u : 0u);
            }
            const uint32_t vbase = smem_u32(sb) + L::KV;
            const int vkey = (lane & 7) + 8 * ((lane >> 3) & 1), vc = lane >> 4;
            if constexpr (Q8) {
                // 16 columns of codes at a time: a transposed 16-bit element is
                // the pair of codes of columns 2 g8, 2 g8 + 1
#pragma unroll
                for (int n = 0; n < 8; n += 2) {
                    uint32_t x[4];
                    ldsm_x4_t(vbase + swz128(vkey, n + vc), x);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t lo = __byte_perm(x[2 * q], 0u, 0x3120), hi = __byte_perm(x[2 * q + 1], 0u, 0x3120);
                        const int nn = 2 * (n + q);
                        mma16<TV>(o[nn], pf[0], pf[1], pf[2], pf[3], codes2<TV>(lo & 0xffffu) & ka,
                                  codes2<TV>(hi & 0xffffu) & kb);
                        mma16<TV>(o[nn + 1], pf[0], pf[1], pf[2], pf[3], codes2<TV>(lo >> 16) & ka,
                                  codes2<TV>(hi >> 16) & kb);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                    uint32_t x[4];
                    ldsm_x4_t(vbase + (n >> 3) * (L::KV / 2) + swz128(vkey, (n & 7) + vc), x);
                    mma16<TV>(o[n], pf[0], pf[1], pf[2], pf[3], x[0] & ka, x[1] & kb);
                    mma16<TV>(o[n + 1], pf[0], pf[1], pf[2], pf[3], x[2] & ka, x[3] & kb);
                }
            }
            __syncwarp();
            fence_proxy_async_smem();
            ++taken;
            issue();
        }

        // ---- merge the warps: common maximum, then outputs in two rounds of
        // four buffers
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(FULL_MASK, l[r], 1);
            l[r] += __shfl_xor_sync(FULL_MASK, l[r], 2);
        }
        __syncthreads();  // the previous item's merge has been read
        if (t4 == 0) {
            *reinterpret_cast<float2 *>(stat(warp, g8)) = make_float2(m[0], l[0]);
            *reinterpret_cast<float2 *>(stat(warp, g8 + 8)) = make_float2(m[1], l[1]);
        }
        __syncthreads();
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float M = NEG_INF;
#pragma unroll
            for (int w = 0; w < SM_WARPS; ++w) M = fmaxf(M, *stat(w, g8 + 8 * r));
            f[r] = m[r] > NEG_INF ? ex2(m[r] - M) : 0.0f;
        }
        float *mine = merge + (warp & 3) * 16 * MROW;
#pragma unroll
        for (int round = 0; round < 2; ++round) {
            if ((warp >> 2) == round) {
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    // columns of this accumulator: 8 n + 2 t4 + {0, 1}, or with codes
                    // 16 (n / 2) + 4 t4 + (n mod 2) + {0, 2}
                    const int d0 = Q8 ? 16 * (n >> 1) + 4 * t4 + (n & 1) : 8 * n + 2 * t4, d1 = d0 + (Q8 ? 2 : 1);
                    float *a = mine + g8 * MROW, *b = a + 8 * MROW;
                    if (round == 0) {
                        a[d0] = o[n][0] * f[0];
                        a[d1] = o[n][1] * f[0];
                        b[d0] = o[n][2] * f[1];
                        b[d1] = o[n][3] * f[1];
                    } else {
                        a[d0] += o[n][0] * f[0];
                        a[d1] += o[n][1] * f[0];
                        b[d0] += o[n][2] * f[1];
                        b[d1] += o[n][3] * f[1];
                    }
                }
            }
            __syncthreads();
        }
        const bool split = t0 > 0 || tn < e.ntiles;
        float *part = p.small.part + (size_t)(2 * c + (first_item && t0 > 0 ? 0 : 1)) * (PG_SROWS * PG_PART);
        for (int r = warp; r < rows; r += SM_WARPS) {  // a warp writes a row
            float M = NEG_INF, Ls = 0.0f;
#pragma unroll
            for (int w = 0; w < SM_WARPS; ++w) M = fmaxf(M, *stat(w, r));
            if (M > NEG_INF) {
#pragma unroll
                for (int w = 0; w < SM_WARPS; ++w) Ls += stat(w, r)[1] * ex2(*stat(w, r) - M);
            }
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * 16 + r) * MROW + 4 * lane);
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            if (split) {
                if (lane == 0) {
                    part[r] = M;
                    part[PG_SROWS + r] = Ls;
                }
                *reinterpret_cast<float4 *>(part + 2 * PG_SROWS + r * D + 4 * lane) = x;
            } else {
                const float inv = Ls > 0.0f ? 1.0f / Ls : 0.0f;
                x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
                T *dst = static_cast<T *>(p.out) +
                         ((size_t)(e.tok0 + r / p.GQ) * p.Hq + (size_t)h * p.GQ + r % p.GQ) * D + 4 * lane;
                *reinterpret_cast<uint2 *>(dst) = pack4<T>(x);
            }
        }
        first_item = false;
        co.t = tn - 1;
        co.left -= tn - t0 - 1;
        if (!co.next(p)) break;
    }
    if (!ok) {  // a copy did not land in time: wait (bounded) for the others before the memory is given up
        for (; taken < issued; ++taken)
            (void)mbar_wait_bounded(&my_bar[taken % L::STAGES], (uint32_t)(taken / L::STAGES) & 1u);
    }
}

template <class T, bool Q8>
cudaError_t launch_small(const PagedAttendParams &p, cudaStream_t stream)
{
    auto kern = paged_small_kernel<T, Q8>;
    constexpr int smem = SmTile<Q8>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.small.G, SM_WARPS * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_plan(const PagedAttendParams &p, cudaStream_t stream)
{
    paged_plan_kernel<<<1, PLAN_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_small(const PagedAttendParams &p0, int q_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAttendParams p = p0;
    const bool q8 = cache_dtype == VQ_E4M3;
    const uint64_t rows = ((uint64_t)p.c.num_pages * p.c.Hkv) << p.c.page_shift;
    if (!encode_tmap_pages(&p.tmk, p.c.k, rows, q8 ? 1 : 2, KB) || !encode_tmap_pages(&p.tmv, p.c.v, rows, q8 ? 1 : 2, KB))
        return cudaErrorInvalidValue;
    if (q_dtype == VQ_F16) return q8 ? launch_small<__half, true>(p, stream) : launch_small<__half, false>(p, stream);
    return q8 ? launch_small<__nv_bfloat16, true>(p, stream) : launch_small<__nv_bfloat16, false>(p, stream);
}

cudaError_t launch_paged_combine(const PagedAttendParams &p, int q_dtype, bool large, cudaStream_t stream)
{
    const dim3 grid(large ? p.large.G : p.small.G, (large ? PG_LROWS : PG_SROWS) / CB_ROWS);
    if (q_dtype == VQ_F16) {
        if (large) paged_combine_kernel<__half, PG_LROWS, 1><<<grid, 128, 0, stream>>>(p);
        else paged_combine_kernel<__half, PG_SROWS, 0><<<grid, 128, 0, stream>>>(p);
    } else {
        if (large) paged_combine_kernel<__nv_bfloat16, PG_LROWS, 1><<<grid, 128, 0, stream>>>(p);
        else paged_combine_kernel<__nv_bfloat16, PG_SROWS, 0><<<grid, 128, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t paged_attend_take_device_error(unsigned *bits, cudaStream_t stream)
{
    *bits = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_pa_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (*bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_pa_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace vq
