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
// Trees of drafts.  The new token i of depth d_i (its number of ancestors among the
// new ones) is at position p = lens[b] - n_b + d_i and sees the earlier tokens of
// the sequence as above, and of the new ones itself and its ancestors, by the same
// rule on their positions.  The new tokens lie in the cache in the order given, so
// these are bits over the last n_b keys: at most 16 of a small item, which its warps
// find by themselves, and PG_TREE_WORDS words a token for the large ones, which the
// plan's launch writes.
//
// 8-bit cache.  With k_j = 2^a_j K_j and v_j = 2^b_j V_j (codes K, V exact in
// fp16 and bf16) the score is 2^a_j (q . K_j), and the exponent of the value is
// folded into the weight: w'_j = 2^(s_j + b_j - M) with M the maximum of
// s_j + b_j, so that w' is at most 1 whatever the exponents, out = sum w'_j V_j
// / sum w'_j 2^-b_j, and the products take codes that were never scaled.  A zero
// value row, which is stored with exponent 0, counts with the least exponent
// (any serves, as V_j = 0): where the other rows are small, M would else follow
// it, and their weights would leave fp16's range.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "tcgen05.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pa_err);

constexpr int D = 128;
constexpr float NEG_INF = -__builtin_huge_valf();

// ---------------------------------------------------------------- the plan

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_NEAR = 2;     // tiles
constexpr int PLAN_ITEM = 3, PLAN_ITEM_Q8 = 4;  // tiles
constexpr int PLAN_KEPT = 1024;  // entries whose sums stay in shared memory

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

// What is merged where CTA c of g starts, in tile t of nt of an item: the parts of
// the item it enters in its middle, if no earlier CTA does so; 0 otherwise.
template <class F> __device__ __forceinline__ int parts_at(F &&first, int g, int c, int t, int nt)
{
    if (t == 0) return 0;
    const long long u = first(c);
    if (t > u - first(c - 1)) return 0;
    int n = 2;
    while (c + n - 1 < g && first(c + n - 1) < u - t + nt) ++n;
    return n;
}

// The masks and depths of the tokens of sequence b, a thread each: up its ancestors
// twice, for its depth and for the bits.  A parent that does not come before its
// token is reported and taken for the last cached token.  (Beside the plan, in its
// launch, and done before it: that takes 8 us with 64 trees of 16, as without.)
__device__ __forceinline__ void tree_masks(const PagedAttendParams &p, int b, int *parent, uint32_t *rows)
{
    int start = 0, n = 0, len = 0;
    (void)sequence(p, b, start, n, len);  // (the plan reports)
    const int i = threadIdx.x, base = len - n;
    n = min(n, PG_TREE_MAX);
    if (i < n) {
        int a = __ldg(p.parents + start + i);
        if (a < -1 || a >= i) {
            atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
            a = -1;
        }
        parent[i] = a;
    }
    __syncthreads();
    if (i >= n) return;
    uint32_t *row = rows + i * PG_TREE_WORDS;
    for (int w = 0; w < PG_TREE_WORDS; ++w) row[w] = 0u;
    int depth = 0;
    for (int a = parent[i]; a >= 0; a = parent[a]) ++depth;
    int up = 0;
    for (int a = i; a >= 0; a = parent[a], ++up)
        if (p.window == 0 || up < p.window || base + depth - up < p.sinks) row[a >> 5] |= 1u << (a & 31);
    p.depth[start + i] = depth;
    uint4 *dst = reinterpret_cast<uint4 *>(p.masks + (size_t)(start + i) * PG_TREE_WORDS);
    for (int w = 0; w < PG_TREE_WORDS / 4; ++w) dst[w] = make_uint4(row[4 * w], row[4 * w + 1], row[4 * w + 2], row[4 * w + 3]);
}

// One CTA: entries of both classes, sequence by sequence, the units before each,
// and where each CTA of the attention kernels starts.  (Trees: a CTA a sequence
// more, for its tokens' masks.)
__global__ void __launch_bounds__(PLAN_THREADS, 1) paged_plan_kernel(const __grid_constant__ PagedAttendParams p)
{
    __shared__ long long ws[32];
    // units before, and tiles of, the first entries of each class (later ones
    // are read back from memory)
    __shared__ long long s_base[2][PLAN_KEPT];
    __shared__ int s_nt[2][PLAN_KEPT];
    __shared__ long long s_first[PLAN_CTAS + 1];  // first unit of each share
    __shared__ int4 s_at[PLAN_CTAS + 1];          // its entry, head, tile
    pg_go();
    if (blockIdx.x > 0) {
        static_assert(PG_TREE_MAX * PG_TREE_WORDS <= 4 * PLAN_KEPT && PG_TREE_MAX <= 2 * PLAN_KEPT, "room for a tree");
        tree_masks(p, (int)blockIdx.x - 1, s_nt[0], reinterpret_cast<uint32_t *>(s_base));
        return;
    }
    const int lane = threadIdx.x & 31;
    long long carry = 0;  // entries so far: small in the low half, large in the high one
    for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
        const int b = b0 + (threadIdx.x >> 5) + 32 * lane;  // (few sequences: a warp each)
        int start = 0, n = 0, len = 0;
        const int sense = b < p.B ? sequence(p, b, start, n, len) : SEQ_OK;
        if (sense != SEQ_OK) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        // Sequences that do not go back share no token, so their entries fit.  Others
        // could have any number of entries: none of them is planned.
        if (__syncthreads_or(sense == SEQ_BACK)) break;
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
            const int at = first_ + i;  // below pl.cap
            const PgEntry e = make_entry(p, b_, start_, n_, len_, pl.tq, i);
            pl.ent[at] = e;
            if (at < PLAN_KEPT) s_nt[large_][at] = e.ntiles;
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
    if (p.wbase) {  // the units of weighing: two key tiles, a head, a part of the query rows
        long long units = 0;
        bool back = false;
        for (int b0 = 0; b0 < p.B && !back; b0 += PLAN_THREADS) {
            const int b = b0 + threadIdx.x;
            int start = 0, n = 0, len = 0;
            const int sense = b < p.B ? sequence(p, b, start, n, len) : SEQ_OK;
            back = __syncthreads_or(sense == SEQ_BACK);
            long long u = 0, all;
            if (n * p.GQ > p.small_rows) u = (long long)((make_entry(p, b, start, n, len, n, 0).ntiles + 1) / 2) * p.Hkv * pg_parts(p, n);
            const long long before = block_scan(u, ws, all);
            if (b < p.B) p.wbase[b] = units + before;
            units += all;
        }
        if (threadIdx.x == 0) p.wbase[p.B] = back ? 0 : units;
    }
    for (int k = 0; k < 2; ++k) {
        const PgPlan &pl = k ? p.large : p.small;
        if (pl.cap == 0) continue;
        const int nent = (int)(k ? carry >> 32 : carry & 0xffffffffLL);
        auto tiles = [&](int i) { return i < PLAN_KEPT ? s_nt[k][i] : pl.ent[i].ntiles; };
        auto base = [&](int i) { return i < PLAN_KEPT ? s_base[k][i] : pl.base[i]; };
        long long total = 0;
        for (int i0 = 0; i0 < nent; i0 += PLAN_THREADS) {
            const int i = i0 + threadIdx.x;
            const long long u = i < nent ? (long long)tiles(i) * p.Hkv : 0;
            long long all;
            const long long before = block_scan(u, ws, all);
            if (i < nent) {
                if (i < PLAN_KEPT) s_base[k][i] = total + before;
                else pl.base[i] = total + before;
            }
            total += all;
        }
        __syncthreads();
        // Shares of large items are even in cost: a tile is one, and an item costs as
        // much as `item` tiles besides (its first products wait for queries, keys
        // and a softmax, and it writes its output): the times of the chunk kernel's
        // CTAs fit 1.5 us a tile and 5.0 a run of an item over a 16-bit cache, 1.8
        // and 7.3 over codes.
        const int item = k ? (p.c.ke ? PLAN_ITEM_Q8 : PLAN_ITEM) : 0;
        auto cost = [&](int i) { return base(i) + (long long)i * item * p.Hkv; };  // before entry i
        Shares sh;
        sh.set(total + (long long)nent * item * p.Hkv, (int)min((long long)pl.G, total));
        // Where each share starts.  A share of large items moves to the start of an
        // item that is at most PLAN_NEAR tiles away: an item cut in two costs its
        // partial results (2 x 133 KB written and read) and a second start.  With
        // shares even in tiles (item 0) and none moved: three chunks of 300 to 1000
        // tokens 162 us, a mixed step over codes 164, one of 12 chunks in 32
        // sequences 472; with item 3 or 4 and NEAR 2: 155, 152, 419; with NEAR 3:
        // 156, 151, 419, but a window of 4096 231 us against 224.
        for (int c = threadIdx.x; c <= sh.g; c += PLAN_THREADS) {
            const long long x = sh.first(c);
            long long u = total;
            int4 at = make_int4(0, 0, 0, 0);
            if (c < sh.g) {
                int a = 0, z = nent - 1;  // the last entry that starts at or before x
                while (a < z) {
                    const int mid = (a + z + 1) >> 1;
                    if (cost(mid) <= x) a = mid;
                    else z = mid - 1;
                }
                const int nt = tiles(a);
                const long long r = x - cost(a), one = (long long)item + nt;
                const int h = (int)(r / one);
                at = make_int4(a, h, max(0, (int)(r - h * one) - item), 0);
                u = base(a) + (long long)h * nt + at.z;
                if (k && at.z > 0 && at.z <= PLAN_NEAR) {
                    u -= at.z;
                    at.z = 0;
                } else if (k && at.z > 0 && nt - at.z <= PLAN_NEAR) {
                    u += nt - at.z;
                    at.z = 0;
                    if (++at.y == p.Hkv) {
                        at.y = 0;
                        ++at.x;  // (past the last entry: an empty share)
                    }
                }
            }
            s_first[c] = u;
            s_at[c] = at;
        }
        __syncthreads();
        auto first = [&](int c) { return s_first[c]; };
        for (int c = threadIdx.x; c < pl.G; c += PLAN_THREADS) {
            PgStart st = {};
            int4 m = make_int4(0, 0, 0, 0);
            if (c < sh.g && first(c + 1) > first(c)) {
                const int4 at = s_at[c];
                st.ei = at.x;
                st.h = at.y;
                st.t = at.z;
                st.left = (int)(first(c + 1) - first(c));
                st.e = pl.ent[at.x];
                m = make_int4(parts_at(first, sh.g, c, st.t, st.e.ntiles), st.e.tok0, st.e.nt, st.h);
            }
            pl.start[c] = st;
            pl.cmb[c] = m;
        }
        __syncthreads();
    }
    if (p.planned && threadIdx.x == 0) pg_release(p.planned, p.call);
}

// ------------------------------------------------------- the merge of parts

constexpr int CB_WARPS = 8;
constexpr int CB_LARGE = 2;  // rows of a warp: large items (few parts, many rows; 4 rows and two blocks an SM: 1.5 us more)
static_assert(PG_LROWS % (CB_WARPS * CB_LARGE) == 0 && PG_SROWS % CB_WARPS == 0, "whole blocks");

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

// Rows r0, r0 + 1, ..., R of them, of the item merged where CTA c starts, by one
// warp: its parts are the second slot of CTA c - 1 and the first slots of c,
// c + 1, ..., taken in that order on every run, NP at a time with all loads in
// flight (8 of 512 bytes a warp), the maximum followed online.
template <class T, int ROWS, int RT, int R, int NP>
__device__ __forceinline__ void merge_rows(const PagedAttendParams &p, const float *parts_base, int c, int4 at, int r0)
{
    const int lane = threadIdx.x & 31, parts = at.x;
    const int tqt = RT / p.GQ;  // tokens of a query tile of RT rows
    constexpr size_t SLOT = (size_t)ROWS * PG_PART;
    const float *first = parts_base + (size_t)(2 * c - 1) * SLOT;
    float M[R], L[R];
    float4 O[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        M[j] = NEG_INF;
        L[j] = 0.0f;
        O[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int k0 = 0; k0 < parts; k0 += NP) {
        float m[R][NP], l[R][NP];
        float4 o[R][NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int k = min(k0 + i, parts - 1);
            const float *s = first + (size_t)(2 * k - (k > 0 ? 1 : 0)) * SLOT + r0;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                m[j][i] = s[j];
                l[j][i] = s[ROWS + j];
                const int r = r0 + j, at4 = ROWS == PG_LROWS ? (r & ~31) * D + (lane >> 1) * 256 + (r & 31) * 8 + (lane & 1) * 4
                                                             : r * D + 4 * lane;
                o[j][i] = *reinterpret_cast<const float4 *>(s - r0 + 2 * ROWS + at4);
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float N = M[j];
#pragma unroll
            for (int i = 0; i < NP; ++i) N = fmaxf(N, m[j][i]);
            if (N == NEG_INF) continue;  // nothing seen so far
            const float f0 = ex2(M[j] - N);
            M[j] = N;
            L[j] *= f0;
            O[j].x *= f0; O[j].y *= f0; O[j].z *= f0; O[j].w *= f0;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float f = k0 + i < parts ? ex2(m[j][i] - N) : 0.0f;
                L[j] = fmaf(l[j][i], f, L[j]);
                O[j].x = fmaf(o[j][i].x, f, O[j].x);
                O[j].y = fmaf(o[j][i].y, f, O[j].y);
                O[j].z = fmaf(o[j][i].z, f, O[j].z);
                O[j].w = fmaf(o[j][i].w, f, O[j].w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int r = r0 + j, half = r / RT, rr = r % RT;
        const int tok = half * tqt + rr / p.GQ, g = rr % p.GQ;
        if (rr >= tqt * p.GQ || tok >= at.z) continue;  // a row of no token
        const float inv = L[j] > 0.0f ? 1.0f / L[j] : 0.0f;
        const size_t qrow = (size_t)(at.y + tok) * p.Hq + (size_t)at.w * p.GQ + g;
        if (p.lse && lane == 0) p.lse[pg_lse_at(p, at.y + tok, at.w, g)] = pg_lse(M[j], L[j]);
        T *dst = static_cast<T *>(p.out) + qrow * D + 4 * lane;
        *reinterpret_cast<uint2 *>(dst) =
            pack4<T>(make_float4(O[j].x * inv, O[j].y * inv, O[j].z * inv, O[j].w * inv));
    }
}

// Blocks x: the CTAs at whose start an item may have to be merged; blocks y: rows
// of large items, then of small ones.
template <class T>
__global__ void __launch_bounds__(32 * CB_WARPS, 4) paged_combine_kernel(const __grid_constant__ PagedAttendParams p)
{
    pg_go();
    pg_wait();
    if (p.planned && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.planned = 0;  // (a graph repeats the call's number)
    const int first_small = p.large.cap ? PG_LROWS / (CB_WARPS * CB_LARGE) : 0;
    const int c = blockIdx.x, y = blockIdx.y, warp = threadIdx.x >> 5;
    if (y < first_small) {
        const int4 at = p.large.cmb[c];
        const int r0 = (y * CB_WARPS + warp) * CB_LARGE, tqt = 128 / p.GQ;
        // (rows past the item's tokens come in whole query tiles, or at its end)
        if (at.x > 0 && (r0 < 128 ? r0 / p.GQ < at.z : tqt + (r0 - 128) / p.GQ < at.z))
            merge_rows<T, PG_LROWS, 128, CB_LARGE, 2>(p, p.large.part, c, at, r0);
    } else {
        const int4 at = p.small.cmb[c];
        const int r0 = (y - first_small) * CB_WARPS + warp;
        if (at.x > 0 && r0 < at.z * p.GQ) merge_rows<T, PG_SROWS, PG_SROWS, 1, 8>(p, p.small.part, c, at, r0);
    }
}

// --------------------------------------------------------- the small kernel
//
// HBM bounds this kernel: every visible key and value is read once per kv head
// for all of its query rows (at most 8 NT).  One CTA per SM: two warps copy
// tiles of 128 keys (one the keys, one the values) into a ring by TMA, a box
// per page; the others compute, each on 16 of a tile's keys with a running
// maximum, sum and output of its own in registers, in groups of 8 that take the
// tiles in turn.  What bounds a warp is the latency of its chain (wait, scores,
// maximum, weights, product), so the copies' page lookups and waits are not in
// it, and over codes, which take more work a byte, two groups hide one another's.
//
// Both products are 16 x 8 x 16 mma.sync with the cache as the 16-row operand:
// S^T = K Q^T and O^T += V^T W^T, the query rows in the 8-wide dimension, where
// little is padding (a tile of 128 tensor-memory rows would be mostly padding).
// The order of the 128 coordinates in the score product is free as long as both
// operands share it: a lane takes 16 consecutive bytes of a cache row per load,
// for 16-bit entries and for codes alike.
constexpr int KB = 16;         // keys of a warp's block
constexpr float OFF = 7.0f;    // weights reach up to 2^(OFF + LAG): fp16 stays normal down to 2^-14
constexpr float LAG = 8.0f;    // the maximum is only followed when it grew by more than this

template <bool Q8, int NT> struct SmShape {
    static constexpr int ROW = Q8 ? 128 : 256;            // bytes of a cache row
    static constexpr int KV = PG_TILE * ROW;              // keys, or values, of a tile
    static constexpr int STAGE = 2 * KV;
    static constexpr int STAGES = Q8 ? 6 : 3;
    static constexpr int EXP = Q8 ? 2 * PG_TILE : 0;      // exponents of a tile
    // Groups of 8 warps: two over codes, which take more work a byte.  A warp
    // waits only for its own group's tiles, so a ring slot has to come back to
    // the same group: another group's pass in between would be taken for the
    // next one (the parity of a barrier tells two passes apart, not three).
    static constexpr int GROUPS = NT == 1 && Q8 ? 2 : 1;
    static_assert(STAGES % GROUPS == 0, "a slot belongs to one group");
    static constexpr int WARPS = 8 * GROUPS;              // that compute
    static constexpr int PAIRS = GROUPS;                  // of warps that copy: keys and values; they take the tiles in turn
    static_assert(STAGES % PAIRS == 0, "a slot belongs to one pair");
    static constexpr int THREADS = 32 * (WARPS + 2 * PAIRS);
    static constexpr int ROWS = 8 * NT;
    static constexpr int MBUF = NT == 1 ? 4 : 2;          // buffers that the warps' outputs are summed in
    static constexpr int MROW = D + 4;                    // row of a buffer (floats)
    static constexpr int SMEM = 1024 + STAGES * (STAGE + EXP + 16) + MBUF * ROWS * MROW * 4 + WARPS * ROWS * 8;
};
static_assert(SmShape<false, 1>::SMEM <= 232448 && SmShape<true, 1>::SMEM <= 232448 &&
                  SmShape<false, 2>::SMEM <= 232448 && SmShape<true, 2>::SMEM <= 232448,
              "shared memory of one CTA");

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 8 x 8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// The plan of a call whose sequences are all small, made by every CTA for itself
// (a kernel for it cost a launch, 4 us before the first copy): the start of CTA c
// into `ws` as a PgStart, what is merged there into the plan's cmb.  Entries are
// the sequences with new tokens, `ei` the sequence.
template <int THREADS> __device__ __forceinline__ void own_plan(const PagedAttendParams &p, int c, long long *ws)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PgStart *out = reinterpret_cast<PgStart *>(ws);
    long long *sums = ws + 8;
    const int per = (p.B + THREADS - 1) / THREADS, b0 = threadIdx.x * per, b1 = min(b0 + per, p.B);
    long long mine = 0;
    bool fits = true;
    for (int b = b0; b < b1; ++b) {
        int start, n, len;
        fits = sequence(p, b, start, n, len) == SEQ_OK && fits;
        if (n > 0) mine += (long long)make_entry(p, b, start, n, len, p.small.tq, 0).ntiles * p.Hkv;
    }
    if (!fits && c == 0) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
    long long x = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, x, s);
        if (lane >= s) x += y;
    }
    if (lane == 31) sums[warp] = x;
    if (threadIdx.x == 0) out->left = 0;
    __syncthreads();
    long long base = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += sums[w];
        total += sums[w];
    }
    Shares sh;
    sh.set(total, p.small.G);
    int4 m = make_int4(0, 0, 0, 0);
    if (c < sh.g) {
        const long long u = sh.first(c);
        if (u >= base && u < base + mine) {  // one thread: the share starts in its sequences
            for (int b = b0; b < b1; ++b) {
                int start, n, len;
                (void)sequence(p, b, start, n, len);
                if (n == 0) continue;
                const PgEntry e = make_entry(p, b, start, n, len, p.small.tq, 0);
                if (u < base + (long long)e.ntiles * p.Hkv) {
                    PgStart st;
                    const int r = (int)(u - base);
                    st.ei = b;
                    st.h = r / e.ntiles;
                    st.t = r - st.h * e.ntiles;
                    st.left = (int)(sh.first(c + 1) - u);
                    st.e = e;
                    *out = st;
                    p.small.cmb[c] = make_int4(
                        parts_at([&](int i) { return sh.first(i); }, sh.g, c, st.t, e.ntiles), e.tok0, e.nt, st.h);
                    break;
                }
                base += (long long)e.ntiles * p.Hkv;
            }
        }
    } else if (threadIdx.x == 0) {
        p.small.cmb[c] = m;
    }
    __syncthreads();
}

// Whether the plan kernel's plan is there.  It is, from the start: the small kernel
// runs when the large kernel's CTAs do, which have waited for the plan.  But only
// they have: this grid waits for the large kernel at its end.  So what it reads of
// the plan is ordered by this acquire and the plan's release, not by that wait
// (waiting first took 4 to 15 % more of a mixed step's time).
__device__ __forceinline__ bool planned(const PagedAttendParams &p)
{
    const uint64_t t0 = globaltimer_ns();
    while (pg_acquire(p.planned) != p.call) {
        if (globaltimer_ns() - t0 > MBAR_TIMEOUT_NS) {
            atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
            return false;
        }
    }
    return true;
}

// T: query and output type; Q8: e4m3 cache (values are then taken as fp16)
template <class T, bool Q8, int NT, int MODE>
__global__ void __launch_bounds__(SmShape<Q8, NT>::THREADS, 1) paged_small_kernel(const __grid_constant__ PagedAttendParams p)
{
    using L = SmShape<Q8, NT>;
    using TV = typename std::conditional<Q8, __half, T>::type;  // operand type of both products
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *stages = smem_1k(smem_raw);
    float *merge = reinterpret_cast<float *>(stages + L::STAGES * L::STAGE);
    float2 *stat = reinterpret_cast<float2 *>(merge + L::MBUF * L::ROWS * L::MROW);  // [warp][row] maximum, sum
    unsigned char *exps = reinterpret_cast<unsigned char *>(stat + L::WARPS * L::ROWS);
    uint64_t *full = reinterpret_cast<uint64_t *>(exps + L::STAGES * L::EXP), *empty = full + L::STAGES;

    const int c = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 8);
        }
        fence_mbar_init();
    }
    // Alone, this kernel makes its own plan.  After the large kernel it has that
    // of the plan kernel, and waits at its end for the large kernel, so that the
    // merge after it comes after both.
    const bool alone = p.large.cap == 0;
    pg_go();
    if (!__syncthreads_and(alone || threadIdx.x != 0 || planned(p))) {
        pg_wait();
        return;
    }
    PgRun r;
    if (alone) {
        own_plan<L::THREADS>(p, c, reinterpret_cast<long long *>(merge));
        r.start(*reinterpret_cast<const PgStart *>(merge));
        __syncthreads();
    } else {
        r.start(p.small.start[c]);
    }
    if (r.left <= 0) {
        if (!alone) pg_wait();
        return;
    }
    // the next entry: in a plan's list, or the next sequence with new tokens
    auto step = [&](PgRun &x) {
        ++x.ei;
        if (!alone) {
            x.e = pg_entry(p.small.ent + x.ei);
            return;
        }
        int start = 0, n = 0, len = 0;
        for (; x.ei < p.B; ++x.ei) {
            (void)sequence(p, x.ei, start, n, len);
            if (n > 0) break;
        }
        x.e = make_entry(p, x.ei, start, n, len, p.small.tq, 0);
    };
    PgRing<L::STAGES> ring;

    if (warp >= L::WARPS) {
        // ------------------------------------------------ copies: keys, values
        const int pair = (warp - L::WARPS) >> 1;
        const bool val = ((warp - L::WARPS) & 1) != 0;
        const CUtensorMap *map = val ? &p.tmv : &p.tmk;
        const uint8_t *ex = val ? p.c.ve : p.c.ke;
        const int box = min(1 << p.c.page_shift, PG_TILE), nbox = PG_TILE / box;
        const uint64_t pol = l2_policy_evict_first();
        int tiles = 0, last = -1;  // tiles of the CTA before this run; this pair's last one
        bool ok = true;
        do {
            PgView view;
            view.set(r.e, p.window, p.sinks);
            // a lane per box: its page is looked up two tiles ahead
            auto row_of = [&](int t) -> int {  // -1: nothing to copy, -2: no such page
                if (t >= r.tn || lane >= nbox) return -1;
                const int k = pg_tile_key(r.e, t) + lane * box;
                if (!view.any(k, k + box)) return -1;
                const int lp = k >> p.c.page_shift;
                const int page = lp < p.max_pages ? __ldg(p.table + (long long)r.e.b * p.max_pages + lp) : -1;
                if (page < 0 || page >= p.c.num_pages) return -2;
                return ((page * p.c.Hkv + r.h) << p.c.page_shift) + (k & ((1 << p.c.page_shift) - 1));
            };
            // the exponents of this lane's four keys, one tile ahead (a copy of 16
            // bytes takes the TMA unit as long as one of 2 KB)
            auto exps_of = [&](int row) -> uint32_t {
                if constexpr (!Q8) return 0u;
                const int k = 4 * lane, rw = __shfl_sync(FULL_MASK, row, k / box);
                return rw >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(ex + rw + k % box)) : PG_EXP0;
            };
            // the same four, zero value rows with the least exponent
            auto exps_used = [&](int row, uint32_t x) -> uint32_t {
                if (!val || !__any_sync(FULL_MASK, __vcmpeq4(x, PG_EXP0) != 0u)) return x;
                const int k = 4 * lane, rw = __shfl_sync(FULL_MASK, row, k / box);
                return rw >= 0 ? pg_value_exps(x, static_cast<const unsigned char *>(p.c.v) + (long long)(rw + k % box) * D) : x;
            };
            int mine = r.t0;  // this pair's first tile of the run
            if (L::PAIRS > 1 && (tiles & 1) != pair) {
                ++mine;
                ring.step();
            }
            int row1 = row_of(mine), row2 = row_of(mine + L::PAIRS);
            uint32_t x1 = exps_of(row1);
            for (int t = mine; t < r.tn && ok; t += L::PAIRS) {
                const int row = row1;
                const uint32_t x = x1;
                row1 = row2;
                row2 = row_of(t + 2 * L::PAIRS);
                x1 = exps_of(row1);
                if (row < -1) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
                if (tiles + (t - r.t0) >= L::STAGES) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&empty[ring.s], ring.par ^ 1u));
                if (!ok) {
                    if (lane == 0) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
                    break;
                }
                // boxes of a missing page are left as they are: reported, their
                // keys' scores are not specified
                const unsigned held = __ballot_sync(FULL_MASK, row >= 0);
                unsigned char *dst = stages + ring.s * L::STAGE + (val ? L::KV : 0);
                uint64_t *bar = &full[ring.s];
                if constexpr (Q8) {
                    reinterpret_cast<uint32_t *>(exps + ring.s * L::EXP + (val ? PG_TILE : 0))[lane] = exps_used(row, x);
                    __syncwarp();
                }
                if (elect_lane()) mbar_arrive_expect_tx(bar, (uint32_t)(__popc(held) * box * L::ROW));
                __syncwarp();
                if (row >= 0) {  // a lane per box
                    if constexpr (Q8) tma_load_2d(dst + lane * box * L::ROW, map, 0, row, bar, pol);
                    else tma_load_3d(dst + lane * box * L::ROW, map, 0, row, 0, bar, pol);
                }
                __syncwarp();
                ring.step();
                // (past the other pair's tile, if the run has one more)
                if (L::PAIRS > 1 && t + 1 < r.tn) ring.step();
                last = tiles + (t - r.t0);
            }
            tiles += r.tn - r.t0;
        } while (ok && r.next(p.Hkv, step));
        // every copy of this pair has landed before the CTA may exit
        for (int j = last; j >= 0 && j > last - L::STAGES; j -= L::PAIRS) {
            (void)mbar_wait_bounded(&full[j % L::STAGES], (uint32_t)(j / L::STAGES) & 1u);
        }
        if (!alone) pg_wait();
        return;
    }

    // ---------------------------------------------------- scores, softmax, values
    const int group = warp >> 3, g8 = lane >> 2, t4 = lane & 3;
    const int kw = KB * (warp & 7);  // this warp's keys of a tile
    // a box lies in its 128-byte columns one after another: one for codes, two
    // halves for 16-bit entries
    const int box = min(1 << p.c.page_shift, PG_TILE), half = box * 128;
    const int at = (kw / box) * box * L::ROW + (kw % box) * 128;
    int tile = 0;                    // tiles of this CTA so far: group g takes those with tile mod GROUPS == g
    bool ok = true;
    do {
        const PgEntry &e = r.e;
        PgView v;
        v.set(e, p.window, p.sinks);
        const int rows = e.nt * p.GQ;
        // query fragments: row 8 nt + g8 of the item; this lane's coordinates
        // are those of its 16-byte pieces of a cache row (8 entries or 16 codes)
        uint32_t qf[NT][16];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + g8;
            const bool in = row < rows;
            const T *src = static_cast<const T *>(p.q);
            if (in) src += (e.tok0 + row / p.GQ) * p.qst + ((long long)r.h * p.GQ + row % p.GQ) * p.qsh;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = Q8 ? 16 * (t4 + 4 * (j >> 1)) + 8 * (j & 1) : 8 * (t4 + 4 * j);
                const uint4 w = in ? __ldg(reinterpret_cast<const uint4 *>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
                qf[nt][4 * j] = w.x;
                qf[nt][4 * j + 1] = w.y;
                qf[nt][4 * j + 2] = w.z;
                qf[nt][4 * j + 3] = w.w;
            }
        }
        // Over codes the operands are fp16, which one instruction makes of a pair
        // of codes (bf16 takes five): bf16 queries become fp16 by a power of two
        // for each row that brings its largest entry to [2^14, 2^15): exact but
        // for entries 2^-28 of that and below.
        float back_q[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) back_q[i] = 1.0f;
        if constexpr (Q8 && std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t top = 0u;
#pragma unroll
                for (int j = 0; j < 16; ++j) top = __vmaxu2(top, qf[nt][j] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(FULL_MASK, top, 1));
                top = max(top, __shfl_xor_sync(FULL_MASK, top, 2));
                const int e = max((int)(top >> 7) - 127, -100);
                const float f = pow2f(14 - e);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qf[nt][j]));
                    qf[nt][j] = pack2<__half>(v.x * f, v.y * f);
                }
                const float b = pow2f(e - 14);  // of row 8 nt + g8; wanted of rows 8 nt + 2 t4 + {0, 1}
#pragma unroll
                for (int i = 0; i < 2; ++i) back_q[2 * nt + i] = __shfl_sync(FULL_MASK, b, 4 * (2 * t4 + i));
            }
        }
        // the rows of this lane's results are 8 nt + 2 t4 + {0, 1}; their
        // visible keys: j <= pos, and the window
        int pos[2 * NT], low[2 * NT];
        [[maybe_unused]] uint32_t draft[2 * NT];  // (trees) the new tokens that the row sees; pos: the keys before them
        if constexpr (MODE == PG_TREE) {
            int parent = lane < e.nt ? __ldg(p.parents + e.tok0 + lane) : -1;
            if (parent < -1 || parent >= lane) {
                atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
                parent = -1;
            }
            int depth = 0, up = 0;
            uint32_t mask = 0u;
            for (int a = parent; __any_sync(FULL_MASK, a >= 0);) {
                const int next = __shfl_sync(FULL_MASK, parent, max(a, 0));
                depth += a >= 0 ? 1 : 0;
                a = a >= 0 ? next : -1;
            }
            for (int a = lane; __any_sync(FULL_MASK, a >= 0); ++up) {
                const int next = __shfl_sync(FULL_MASK, parent, max(a, 0));
                if (a >= 0 && (p.window == 0 || up < p.window || e.p0 + depth - up < p.sinks)) mask |= 1u << a;
                a = a >= 0 ? next : -1;
            }
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int row = 8 * (i >> 1) + 2 * t4 + (i & 1), tok = row / p.GQ;
                const int d = __shfl_sync(FULL_MASK, depth, tok);
                const uint32_t mk = __shfl_sync(FULL_MASK, mask, tok);
                pos[i] = row < rows ? e.p0 - 1 : -1;
                low[i] = p.window > 0 ? e.p0 + d - p.window + 1 : 0;
                draft[i] = row < rows ? mk : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int row = 8 * (i >> 1) + 2 * t4 + (i & 1);
                pos[i] = row < rows ? e.p0 + row / p.GQ : -1;
                low[i] = p.window > 0 ? pos[i] - p.window + 1 : 0;
            }
        }
        const int lo_all = p.window > 0 ? e.p0 + e.nt - p.window : 0;  // the last row's first key in the window
        [[maybe_unused]] float *scores = nullptr;  // (WEIGH) of this lane's first row and key
        if constexpr (MODE == PG_WEIGH) scores = p.scores + (((size_t)e.b * p.Hkv + r.h) * p.srows + 2 * t4) * p.keys + g8;
        float m[2 * NT], l[2 * NT], o[NT][8][4];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            m[i] = NEG_INF;
            l[i] = 0.0f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][n][j] = 0.0f;

        for (int t = r.t0; t < r.tn; ++t, ++tile, ring.step()) {
            if (L::GROUPS > 1 && (tile & 1) != group) continue;
            if (!ok) continue;
            if (!__all_sync(FULL_MASK, mbar_wait_bounded(&full[ring.s], ring.par))) {
                if (lane == 0) atomicOr(&g_pa_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
                ok = false;
                continue;
            }
            const int k0 = pg_tile_key(e, t) + kw;
            if (v.any(k0, k0 + KB)) {
                const unsigned char *sb = stages + ring.s * L::STAGE + at;
                // ---- scores: S^T[key][row]; this lane's keys are g8 and g8 + 8
                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[nt][j] = 0.0f;
                if constexpr (Q8) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 wa = *reinterpret_cast<const uint4 *>(sb + swz128(g8, t4 + 4 * q));
                        const uint4 wb = *reinterpret_cast<const uint4 *>(sb + swz128(g8 + 8, t4 + 4 * q));
                        const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_to_f16x4(xa[j], a0, a2);
                            e4m3x4_to_f16x4(xb[j], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16<TV>(s[nt], a0, a1, a2, a3, qf[nt][8 * q + 2 * j], qf[nt][8 * q + 2 * j + 1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const unsigned char *h = sb + (q >> 1) * half;
                        const uint4 wa = *reinterpret_cast<const uint4 *>(h + swz128(g8, t4 + 4 * (q & 1)));
                        const uint4 wb = *reinterpret_cast<const uint4 *>(h + swz128(g8 + 8, t4 + 4 * (q & 1)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16<T>(s[nt], wa.x, wb.x, wa.y, wb.y, qf[nt][4 * q], qf[nt][4 * q + 1]);
                            mma16<T>(s[nt], wa.z, wb.z, wa.w, wb.w, qf[nt][4 * q + 2], qf[nt][4 * q + 3]);
                        }
                    }
                }
                // ---- scale, mask
                [[maybe_unused]] float raw[NT][4];  // (WEIGH) scores without the values' exponents
                const bool whole = k0 + KB <= e.p0 + (MODE == PG_TREE ? 0 : 1) && (p.window == 0 || k0 >= lo_all || k0 + KB <= v.sink);
                float fa[2] = {p.qscale, p.qscale}, fb[2] = {0.0f, 0.0f}, back[2] = {1.0f, 1.0f};
                if constexpr (Q8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const unsigned char *x = exps + ring.s * L::EXP + kw + g8 + 8 * i;
                        const int a = (int)x[0] - 127, b = (int)x[PG_TILE] - 127;
                        fa[i] *= pow2f(max(a, -126));
                        fb[i] = (float)b;
                        back[i] = pow2f(max(-b, -126));
                    }
                }
                uint32_t pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = s[nt][j] * back_q[2 * nt + (j & 1)];
                        if constexpr (MODE == PG_WEIGH) raw[nt][j] = x * fa[Q8 ? j >> 1 : 0];
                        s[nt][j] = Q8 ? fmaf(x, fa[j >> 1], fb[j >> 1]) : s[nt][j] * fa[0];
                    }
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = k0 + g8 + 8 * (j >> 1), i = 2 * nt + (j & 1);
                            bool in = k <= pos[i] && (k >= low[i] || k < v.sink);
                            if constexpr (MODE == PG_TREE) in = in || ((unsigned)(k - e.p0) < 32u && (draft[i] >> (k - e.p0)) & 1u);
                            s[nt][j] = in ? s[nt][j] : NEG_INF;
                            if constexpr (MODE == PG_WEIGH) raw[nt][j] = in ? raw[nt][j] : NEG_INF;
                        }
                    }
                    if constexpr (MODE == PG_WEIGH) {
                        // [row][key]: a store of the warp fills whole sectors (keys lie in
                        // order along g8, four rows along t4)
                        float *at = scores + (size_t)(8 * nt) * p.keys + k0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (8 * nt + 2 * t4 + i < rows) {
                                at[(size_t)i * p.keys] = raw[nt][i];
                                at[(size_t)i * p.keys + 8] = raw[nt][i + 2];
                            }
                        }
                    }
                    // ---- softmax: a row's 16 scores lie in the 8 lanes of one t4
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(s[nt][i], s[nt][i + 2]);
#pragma unroll
                        for (int sh = 4; sh <= 16; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, sh));
                        float &mi = m[2 * nt + i];
                        if (x - OFF > mi + LAG) {
                            const float f = ex2(mi - (x - OFF));
                            mi = x - OFF;
                            l[2 * nt + i] *= f;
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                o[nt][n][i] *= f;
                                o[nt][n][i + 2] *= f;
                            }
                        }
                    }
                    const float ma = m[2 * nt] > NEG_INF ? m[2 * nt] : 0.0f, mb = m[2 * nt + 1] > NEG_INF ? m[2 * nt + 1] : 0.0f;
                    const float w0 = ex2(s[nt][0] - ma), w1 = ex2(s[nt][1] - mb), w2 = ex2(s[nt][2] - ma),
                                w3 = ex2(s[nt][3] - mb);
                    if constexpr (Q8) {
                        l[2 * nt] = fmaf(w0, back[0], fmaf(w2, back[1], l[2 * nt]));
                        l[2 * nt + 1] = fmaf(w1, back[0], fmaf(w3, back[1], l[2 * nt + 1]));
                    } else {
                        l[2 * nt] += w0 + w2;
                        l[2 * nt + 1] += w1 + w3;
                    }
                    // W^T as the second operand: [key][row] to [row][key pairs]
                    pf[nt][0] = transpose8(pack2<TV>(w0, w1));
                    pf[nt][1] = transpose8(pack2<TV>(w2, w3));
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
                if constexpr (Q8) {
                    // 16 columns of codes at a time: a transposed 16-bit element is
                    // the pair of codes of columns 2 g8, 2 g8 + 1, which become
                    // rows g8 and g8 + 8 of the operand
                    const int vkey = (lane & 7) + 8 * ((lane >> 3) & 1), vc = lane >> 4;
#pragma unroll
                    for (int n = 0; n < 8; n += 2) {
                        uint32_t x[4];
                        ldsm_x4_t(vbase + swz128(vkey, n + vc), x);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            // (a hidden key's codes become zero: the halves of x are keys here)
                            const uint32_t lo = __byte_perm(x[2 * q] & ka, 0u, 0x3120);
                            const uint32_t hi = __byte_perm(x[2 * q + 1] & kb, 0u, 0x3120);
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_to_f16x4(lo, a0, a1);
                            e4m3x4_to_f16x4(hi, a2, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16<TV>(o[nt][n + q], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                        }
                    }
                } else {
                    const int vkey = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        uint32_t x[4];
                        ldsm_x4_t(vbase + (n >> 2) * half + swz128(vkey, 2 * (n & 3) + vc), x);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16<TV>(o[nt][n], x[0] & ka, x[1] & ka, x[2] & kb, x[3] & kb, pf[nt][0], pf[nt][1]);
                    }
                }
            }
            fence_proxy_async_smem();  // the tile was read; a copy may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[ring.s]);
        }

        // ---- merge the warps: common maximum, then the outputs, MBUF at a time
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1) l[i] += __shfl_xor_sync(FULL_MASK, l[i], sh);
        bar_compute<L::WARPS * 32>();  // the previous item's merge has been read
        if (g8 == 0) {
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i)
                stat[warp * L::ROWS + 8 * (i >> 1) + 2 * t4 + (i & 1)] = make_float2(m[i], l[i]);
        }
        bar_compute<L::WARPS * 32>();
        float f[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            float M = NEG_INF;
#pragma unroll
            for (int w = 0; w < L::WARPS; ++w) M = fmaxf(M, stat[w * L::ROWS + 8 * (i >> 1) + 2 * t4 + (i & 1)].x);
            f[i] = m[i] > NEG_INF ? ex2(m[i] - M) : 0.0f;
        }
        float *mine = merge + (warp % L::MBUF) * L::ROWS * L::MROW;
#pragma unroll 1
        for (int round = 0; round < L::WARPS / L::MBUF; ++round) {
            if (warp / L::MBUF == round) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // coordinate: 16 n + g8 (+ 8), with codes 16 n + 2 g8 (+ 1)
                            const int d = 16 * n + (Q8 ? 2 * g8 + (j >> 1) : g8 + 8 * (j >> 1));
                            float *a = mine + (8 * nt + 2 * t4 + (j & 1)) * L::MROW + d;
                            const float x = o[nt][n][j] * f[2 * nt + (j & 1)];
                            *a = round == 0 ? x : *a + x;
                        }
            }
            bar_compute<L::WARPS * 32>();
        }
        const bool split = r.t0 > 0 || r.tn < e.ntiles;
        float *part = p.small.part + (size_t)(2 * c + (r.first && r.t0 > 0 ? 0 : 1)) * (PG_SROWS * PG_PART);
        for (int row = warp; row < rows; row += L::WARPS) {  // a warp writes a row
            float M = NEG_INF, Ls = 0.0f;
#pragma unroll
            for (int w = 0; w < L::WARPS; ++w) M = fmaxf(M, stat[w * L::ROWS + row].x);
            if (M > NEG_INF) {
#pragma unroll
                for (int w = 0; w < L::WARPS; ++w) Ls += stat[w * L::ROWS + row].y * ex2(stat[w * L::ROWS + row].x - M);
            }
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < L::MBUF; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * L::ROWS + row) * L::MROW + 4 * lane);
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            if (split) {
                if (lane == 0) {
                    part[row] = M;
                    part[PG_SROWS + row] = Ls;
                }
                *reinterpret_cast<float4 *>(part + 2 * PG_SROWS + row * D + 4 * lane) = x;
            } else {
                const float inv = Ls > 0.0f ? 1.0f / Ls : 0.0f;
                x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
                const size_t qrow = (size_t)(e.tok0 + row / p.GQ) * p.Hq + (size_t)r.h * p.GQ + row % p.GQ;
                if (MODE == PG_WEIGH && lane == 0) p.lse[pg_lse_at(p, e.tok0 + row / p.GQ, r.h, row % p.GQ)] = pg_lse(M, Ls);
                T *dst = static_cast<T *>(p.out) + qrow * D + 4 * lane;
                *reinterpret_cast<uint2 *>(dst) = pack4<T>(x);
            }
        }
    } while (r.next(p.Hkv, step));
    if (!alone) pg_wait();
}

template <class T, bool Q8, int NT, int MODE>
cudaError_t launch_small(const PagedAttendParams &p, cudaStream_t stream)
{
    auto kern = paged_small_kernel<T, Q8, NT, MODE>;
    constexpr int smem = SmShape<Q8, NT>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (p.large.cap != 0) return launch_early(kern, dim3(p.small.G), SmShape<Q8, NT>::THREADS, smem, stream, p);
    kern<<<p.small.G, SmShape<Q8, NT>::THREADS, smem, stream>>>(p);  // the call's first kernel
    return cudaGetLastError();
}

template <class T, bool Q8, int MODE>
cudaError_t dispatch_small(const PagedAttendParams &p, cudaStream_t stream)
{
    return p.small_rows <= 8 ? launch_small<T, Q8, 1, MODE>(p, stream) : launch_small<T, Q8, 2, MODE>(p, stream);
}

template <class T, bool Q8>
cudaError_t dispatch_small(const PagedAttendParams &p, cudaStream_t stream)
{
    return p.parents ? dispatch_small<T, Q8, PG_TREE>(p, stream)
           : p.lse   ? dispatch_small<T, Q8, PG_WEIGH>(p, stream)
                     : dispatch_small<T, Q8, PG_CHAIN>(p, stream);
}

}  // namespace

cudaError_t launch_paged_plan(const PagedAttendParams &p, cudaStream_t stream)
{
    paged_plan_kernel<<<p.parents ? 1 + p.B : 1, PLAN_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_small(const PagedAttendParams &p0, int q_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAttendParams p = p0;
    const bool q8 = cache_dtype == VQ_E4M3;
    const uint64_t rows = ((uint64_t)p.c.num_pages * p.c.Hkv) << p.c.page_shift;
    const uint32_t box = 1u << p.c.page_shift < (unsigned)PG_TILE ? 1u << p.c.page_shift : (unsigned)PG_TILE;
    // 16-bit rows as two halves of 64: one copy a box (the TMA unit takes about
    // 47 ns a copy, whatever its size up to 2 KB)
    const bool ok = q8 ? encode_tmap_pages(&p.tmk, p.c.k, rows, 1, box) && encode_tmap_pages(&p.tmv, p.c.v, rows, 1, box)
                       : encode_tmap_halves(&p.tmk, p.c.k, rows, box) && encode_tmap_halves(&p.tmv, p.c.v, rows, box);
    if (!ok) return cudaErrorInvalidValue;
    if (q_dtype == VQ_F16) return q8 ? dispatch_small<__half, true>(p, stream) : dispatch_small<__half, false>(p, stream);
    return q8 ? dispatch_small<__nv_bfloat16, true>(p, stream) : dispatch_small<__nv_bfloat16, false>(p, stream);
}

cudaError_t launch_paged_combine(const PagedAttendParams &p, int q_dtype, cudaStream_t stream)
{
    const dim3 grid(p.large.cap ? p.large.G : p.small.G,
                    (p.large.cap ? PG_LROWS / (CB_WARPS * CB_LARGE) : 0) + (p.small.cap ? PG_SROWS / CB_WARPS : 0));
    return launch_early(q_dtype == VQ_F16 ? paged_combine_kernel<__half> : paged_combine_kernel<__nv_bfloat16>, grid,
                        32 * CB_WARPS, 0, stream, p);
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
