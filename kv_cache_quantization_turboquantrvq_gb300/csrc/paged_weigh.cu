// paged_weigh.cu - the softmax weight that each cached token gets from a call's new
// tokens, added up (sm_103a):
//   a[b][h][j] = sum over the counted tokens i and the query heads g of kv head h of
//                2^(s_igj - lse_ig),   s = scale log2(e) q . k,  lse = log2 sum_j 2^s,
//   weight[j] = (j is a new token ? 0 : decay * weight[j]) + a[j]
// for the keys that some new token sees.  The attention kernels leave lse for every
// query row, and for sequences with few rows the scores themselves: 4 bytes a row
// and key against the key's and value's 512 (or 258) that they read anyway.  For
// chunks the scores are computed once more, here, a tile of 128 keys by 128 query
// rows at a time on the tensor cores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "paged_tc.cuh"
#include "tcgen05.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pw_err);

constexpr float NEG_INF = -__builtin_huge_valf();

// ---------------------------------------------------------------- chunks
//
// The keys are the 128 rows of the product and stay, the query rows are its columns
// and stream through: a thread of the softmax warps holds a key and adds up its row
// of 2^(score - lse) over the columns, without a word to any other thread, and the
// sums need no atomics: a unit is two key tiles of one head against one of at most
// PG_PARTS parts of the query tiles, and writes its own numbers, which the update
// below adds in their order.  (One key tile a unit, its query tiles taken by the two
// groups in turn, asked L2 for 32 KB a product, which takes 512 cycles: as much as
// the SM's path to L2 carries.)
//
// 2048 tokens over 8192, 32 query and 8 kv heads, bf16: 109 us (235 with one key tile a
// unit), 0.92 us for two key tiles against 128 query rows, whose products take 0.54.
// What bounds it is each group's chain of a tile (waits, columns out of tensor memory,
// exponentials), with one warp of a group on a scheduler; a unit costs 1 us besides.
//
// Roles (one CTA per SM): a warp that finds the CTA's units and copies keys and
// queries by TMA, two that issue the products, one that brings the rows' -lse, two
// groups of 4 softmax warps, one for each key tile, with two score tiles each in
// tensor memory; with an 8-bit cache four more warps turn a unit's codes into
// operands of the queries' type (exact in both).  The keys' exponents act on the
// scores, a factor a thread.
template <bool Q8> struct WgShape : WgRings<Q8> {
    using R = WgRings<Q8>;
    using R::KST, R::QST, R::RAW, R::LST, R::IST, R::CONV;
    static constexpr int WARPS = 12 + CONV;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int BARS = 2 * KST + 2 * QST + 2 * RAW + 2 * LST + 2 * IST + 2 * 4 + 1;
    static constexpr int ITEM = 64;            // bytes of a unit's description
    static constexpr int SMEM = 1024 + (KST + QST) * TILE_B + RAW * RAW_B + LST * 128 * 4 + IST * ITEM + 8 * BARS + 16;
};
static_assert(WgShape<false>::SMEM <= 232448 && WgShape<true>::SMEM <= 232448, "shared memory of one CTA");

template <bool Q8> struct WgBars {
    using C = WgShape<Q8>;
    uint64_t *k_full, *k_empty, *q_full, *q_empty, *l_full, *l_empty, *i_full, *i_empty, *s_full, *s_empty, *drain, *raw_full,
        *raw_empty;
    __device__ __forceinline__ explicit WgBars(uint64_t *b)
        : k_full(b), k_empty(k_full + C::KST), q_full(k_empty + C::KST), q_empty(q_full + C::QST), l_full(q_empty + C::QST),
          l_empty(l_full + C::LST), i_full(l_empty + C::LST), i_empty(i_full + C::IST), s_full(i_empty + C::IST),
          s_empty(s_full + 4), drain(s_empty + 4), raw_full(drain + 1), raw_empty(raw_full + C::RAW)
    {
    }
    __device__ __forceinline__ void init()
    {
        for (int s = 0; s < C::KST; ++s) {
            mbar_init(&k_full[s], Q8 ? C::CONV : 1);
            mbar_init(&k_empty[s], C::READERS);
        }
        for (int s = 0; s < C::QST; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], C::READERS);
        }
        for (int s = 0; s < C::LST; ++s) {
            mbar_init(&l_full[s], 1);
            mbar_init(&l_empty[s], 8);
        }
        for (int s = 0; s < C::IST; ++s) {
            mbar_init(&i_full[s], 1);
            mbar_init(&i_empty[s], 3 + 8 + C::CONV);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 4);
        }
        mbar_init(drain, 2);
        for (int s = 0; s < C::RAW; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], C::CONV);
        }
    }
};

// One unit, as the roles read it from shared memory.
struct WgItem {
    int b, h, part;      // b < 0: no more units
    int k0, k1, hi;      // its tiles' first keys (the second -1: there is none), and the end of the sequence's
    int start, n, base;  // the sequence's first query token, new tokens, keys before them
    int i0, qa, qz;      // the first token that counts; query tiles [qa, qz) of those
};

__device__ __forceinline__ WgItem wg_find(const PagedAttendParams &p, long long u)
{
    int a = 0, z = p.B - 1;  // the last sequence that starts at or before u
    while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.wbase[mid] <= u) a = mid;
        else z = mid - 1;
    }
    WgItem w;
    int len;
    (void)sequence(p, a, w.start, w.n, len);
    const PgEntry e = make_entry(p, a, w.start, w.n, len, w.n, 0);
    const int tqt = 128 / p.GQ, parts = pg_parts(p, w.n);
    long long r = u - p.wbase[a];
    w.b = a;
    w.part = (int)(r % parts);
    r /= parts;
    w.h = (int)(r % p.Hkv);
    const int t = 2 * (int)(r / p.Hkv);
    w.k0 = pg_tile_key(e, t);
    w.k1 = t + 1 < e.ntiles ? pg_tile_key(e, t + 1) : -1;
    w.hi = e.hi;
    w.base = e.p0;
    w.i0 = pg_counted(p, w.n);
    // the tokens that may see a key of the tiles: at or behind the first one, and with
    // a window not too far behind the last
    const int sink = p.window > 0 ? min(p.sinks, e.hi) : 0, z1 = max(w.k0, w.k1);
    const long long ia = max(w.i0, w.k0 - w.base);
    long long iz = w.n;
    if (p.window > 0 && w.k0 >= sink) iz = min(iz, (long long)z1 - w.base + PG_TILE - 1 + p.window);
    int qa = 0, cnt = 0;
    if (ia < iz) {
        qa = (int)((ia - w.i0) / tqt);
        cnt = (int)((iz - w.i0 + tqt - 1) / tqt) - qa;
    }
    w.qa = qa + (int)((long long)cnt * w.part / parts);
    w.qz = qa + (int)((long long)cnt * (w.part + 1) / parts);
    return w;
}

// Four codes as two pairs of T, exact.
template <class T> __device__ __forceinline__ void wg_operand(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    e4m3x4_to_f16x4(four, lo, hi);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        lo = ck_pack<__nv_bfloat16>(a.x, a.y);
        hi = ck_pack<__nv_bfloat16>(b.x, b.y);
    }
}

template <class T, bool Q8>
__global__ void __launch_bounds__(WgShape<Q8>::THREADS, 1) paged_weigh_kernel(const __grid_constant__ PagedAttendParams p)
{
    using C = WgShape<Q8>;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *sk = smem_1k(smem_raw);                                  // key tiles
    unsigned char *sq = sk + C::KST * TILE_B;                               // query tiles
    unsigned char *sraw = sq + C::QST * TILE_B;                             // codes
    float *slse = reinterpret_cast<float *>(sraw + C::RAW * RAW_B);         // [LST][128]
    unsigned char *sitem = reinterpret_cast<unsigned char *>(slse + C::LST * 128);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sitem + C::IST * C::ITEM);
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(bars + C::BARS);
    volatile uint32_t *abort_flag = tslot + 1;
    static_assert(sizeof(WgItem) <= C::ITEM, "a unit's description");
    const WgBars<Q8> bar(bars);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tqt = 128 / p.GQ, cols = tqt * p.GQ;
    if (threadIdx.x == 0) {
        WgBars<Q8>(bars).init();
        *abort_flag = 0u;
        fence_mbar_init();
    }
    // columns of query tiles that no copy fills are zeros, not whatever was there
    for (int i = threadIdx.x; i < C::QST * 2 * (128 - cols) * 8; i += C::THREADS) {
        const int c = i & 7, r = (i >> 3) % (128 - cols), t = (i >> 3) / (128 - cols);
        *reinterpret_cast<uint4 *>(sq + t * HALF_B + (cols + r) * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    if (warp == 1) tmem_alloc(const_cast<uint32_t *>(tslot), 512);
    pg_wait();
    pg_go();
    const long long units = p.wbase[p.B];
    qt_fence_before();
    __syncthreads();
    qt_fence_after();
    if (blockIdx.x >= units) {  // the whole CTA
        if (warp == 1) tmem_free(*tslot, 512);
        return;
    }
    const uint32_t tmem = *tslot;

    auto wait = [&](uint64_t *b, uint32_t parity) -> bool {
        if (mbar_try_wait(b, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (mbar_try_wait(b, parity)) return true;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > MBAR_TIMEOUT_NS) {
                atomicOr(&g_pw_err, (unsigned)VQ_DEVERR_WAIT_TIMEOUT);
                *abort_flag = 1u;
                return false;
            }
        }
    };
    bool ok = true;
    auto await = [&](uint64_t *b, uint32_t parity) { ok = ok && __all_sync(FULL_MASK, wait(b, parity)); };
    // Two at a time: asked together first, since one answer after another takes 100
    // cycles each.
    auto await2 = [&](uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb) {
        const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
        if (__all_sync(FULL_MASK, ra && rb)) return;
        await(a, pa);
        await(b, pb);
    };
    // The next unit of a role that is not the first; false: there is none.
    PgRing<C::IST> items;
    auto next = [&](WgItem &w) -> bool {
        await(&bar.i_full[items.s], items.par);
        if (!ok) return false;
        w = *reinterpret_cast<const WgItem *>(sitem + items.s * C::ITEM);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.i_empty[items.s]);
        items.step();
        return w.b >= 0;
    };

    if (warp == 0) {
        // ------------------------------------------------ units, copies (TMA)
        const int box = min(1 << p.c.page_shift, PG_TILE), nbox = PG_TILE / box;
        const int rows_all = p.c.num_pages * p.c.Hkv << p.c.page_shift;  // no box holds this row: reads zeros
        const uint64_t pol = ck_policy();
        PgRing<C::KST> ks;
        PgRing<C::QST> qs;
        [[maybe_unused]] PgRing<C::RAW ? C::RAW : 1> raw;
        int keys = 0, queries = 0;  // tiles copied
        for (long long u = blockIdx.x;; u += gridDim.x) {
            const bool more = u < units;
            WgItem w;
            w.b = -1;
            if (more) w = wg_find(p, u);
            await(&bar.i_empty[items.s], items.par ^ 1u);
            if (!ok) break;
            if (lane == 0) *reinterpret_cast<WgItem *>(sitem + items.s * C::ITEM) = w;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.i_full[items.s]);
            items.step();
            if (!more) break;
            if (w.qa >= w.qz) continue;
            for (int i = 0; i < (w.k1 < 0 ? 1 : 2); ++i) {
                int row = rows_all;
                if (lane < nbox) {
                    const int k = (i ? w.k1 : w.k0) + lane * box;
                    const int lp = k >> p.c.page_shift;
                    const int page = k < w.hi && lp < p.max_pages ? __ldg(p.table + (long long)w.b * p.max_pages + lp) : -1;
                    // (a page that is not there was reported by the attention; its keys are not weighed)
                    if (page >= 0 && page < p.c.num_pages)
                        row = ((page * p.c.Hkv + w.h) << p.c.page_shift) + (k & ((1 << p.c.page_shift) - 1));
                }
                uint64_t *full;
                if constexpr (Q8) {
                    await(&bar.raw_empty[raw.s], raw.par ^ 1u);
                    if (!ok) break;
                    full = &bar.raw_full[raw.s];
                    if (elect_lane()) mbar_arrive_expect_tx(full, RAW_B);
                    __syncwarp();
                    if (lane < nbox) tma_load_2d(sraw + raw.s * RAW_B + lane * box * 128, &p.tmk, 0, row, full, pol);
                    raw.step();
                } else {
                    await(&bar.k_empty[ks.s], ks.par ^ 1u);
                    if (!ok) break;
                    full = &bar.k_full[ks.s];
                    if (elect_lane()) mbar_arrive_expect_tx(full, TILE_B);
                    __syncwarp();
                    if (lane < nbox) {
                        unsigned char *dst = sk + ks.s * TILE_B + lane * box * 128;
                        tma_load_2d(dst, &p.tmk, 0, row, full, pol);
                        tma_load_2d(dst + HALF_B, &p.tmk, 64, row, full, pol);
                    }
                    ks.step();
                }
                ++keys;
                __syncwarp();
            }
            if (!ok) break;
            for (int q = w.qa; q < w.qz; ++q) {
                await(&bar.q_empty[qs.s], qs.par ^ 1u);
                if (!ok) break;
                if (elect_lane()) {
                    mbar_arrive_expect_tx(&bar.q_full[qs.s], (uint32_t)(2 * cols * 128));
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_3d(sq + qs.s * TILE_B + hf * HALF_B, &p.tmq, 64 * hf, w.h * p.GQ, w.start + w.i0 + q * tqt,
                                    &bar.q_full[qs.s], pol);
                }
                __syncwarp();
                qs.step();
                ++queries;
            }
            if (!ok) break;
        }
        // every copy has landed before the CTA may exit
        for (int k = 0; k < C::QST && k < queries; ++k) {
            const int j = queries - 1 - k;
            (void)mbar_wait_bounded(&bar.q_full[j % C::QST], (uint32_t)(j / C::QST) & 1u);
        }
        constexpr int KR = Q8 ? C::RAW : C::KST;
        uint64_t *kb = Q8 ? bar.raw_full : bar.k_full;
        for (int k = 0; k < KR && k < keys; ++k) {
            const int j = keys - 1 - k;
            (void)mbar_wait_bounded(&kb[j % KR], (uint32_t)(j / KR) & 1u);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------ products, a warp a key tile (one
        // for both was busy with waits and issues half of the time)
        constexpr uint32_t ID = ck_idesc(std::is_same<T, __nv_bfloat16>::value, false);
        const uint64_t dk = qt_desc(smem_u32(sk)), dq = qt_desc(smem_u32(sq));
        const uint32_t tm = __shfl_sync(FULL_MASK, tmem, 0);
        const int g = warp >> 1;
        PgRing<C::KST> ks;
        PgRing<C::QST> qs;
        PgRing<C::SST> ss;  // its score tiles
        struct Ops {
            decltype(await) &wait_;
            decltype(await2) &wait2;
            const bool &ok;
            const WgBars<Q8> &bar;
            const uint32_t tm;
            const uint64_t dk, dq;
            const int g;
            __device__ __forceinline__ bool keys(const PgRing<C::KST> &k) const
            {
                wait_(&bar.k_full[k.s], k.par);
                return ok;
            }
            __device__ __forceinline__ bool queries(const PgRing<C::QST> &q) const
            {
                wait_(&bar.q_full[q.s], q.par);
                return ok;
            }
            __device__ __forceinline__ bool both(const PgRing<C::QST> &q, const PgRing<C::SST> &s) const
            {
                wait2(&bar.q_full[q.s], q.par, &bar.s_empty[C::SST * g + s.s], s.par ^ 1u);
                return ok;
            }
            __device__ __forceinline__ void product(const PgRing<C::KST> &k, const PgRing<C::QST> &q, const PgRing<C::SST> &s) const
            {
                qt_fence_after();
                ck_mma_ss(tm + 128 * (C::SST * g + s.s), dk + k.s * (TILE_B >> 4), dq + q.s * (TILE_B >> 4), ID,
                          smem_u32(&bar.s_full[C::SST * g + s.s]));
            }
            __device__ __forceinline__ void used(uint64_t *empty) const
            {
                ck_commit(empty);
                __syncwarp();
            }
            __device__ __forceinline__ void passed(uint64_t *empty) const
            {
                if (elect_lane()) mbar_arrive(empty);
                __syncwarp();
            }
            __device__ __forceinline__ void keys_used(const PgRing<C::KST> &k) const { used(&bar.k_empty[k.s]); }
            __device__ __forceinline__ void keys_passed(const PgRing<C::KST> &k) const { passed(&bar.k_empty[k.s]); }
            __device__ __forceinline__ void queries_used(const PgRing<C::QST> &q) const { used(&bar.q_empty[q.s]); }
            __device__ __forceinline__ void queries_passed(const PgRing<C::QST> &q) const { passed(&bar.q_empty[q.s]); }
        };
        const Ops ops{await, await2, ok, bar, tm, dk, dq, g};
        WgItem w;
        while (next(w)) {
            if (w.qa >= w.qz) continue;
            if (!wg_products(ops, ks, qs, ss, g, w.k1 >= 0, w.qz - w.qa)) break;
        }
        // every product is done before shared and tensor memory are given up
        ck_commit(bar.drain);
        (void)mbar_wait_bounded(bar.drain, 0u);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ the rows' -lse
        uint32_t run = 0u;  // tiles of all units so far
        WgItem w;
        while (next(w)) {
            const int cnt = max(w.qz - w.qa, 0);
            const float *rows = p.lse + ((size_t)w.h * p.T + w.start + w.i0) * p.GQ;
            auto load = [&](int j, float (&x)[4]) {  // (the next tile's while this one waits for its place)
                const int c0 = (w.qa + j) * cols, end = j < cnt ? min(cols, (w.n - w.i0) * p.GQ - c0) : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = 32 * i + lane < end ? -rows[c0 + 32 * i + lane] : NEG_INF;
            };
            float x[4], y[4];
            load(0, x);
            for (int j = 0; j < cnt; ++j) {
                load(j + 1, y);
                const uint32_t at = run + (uint32_t)j;
                const int ls = (int)(at % C::LST);
                await(&bar.l_empty[ls], ((at / C::LST) & 1u) ^ 1u);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    slse[ls * 128 + 32 * i + lane] = x[i];
                    x[i] = y[i];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.l_full[ls]);
            }
            if (!ok) break;
            run += (uint32_t)cnt;
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------ a thread per key
        const int g = (warp - 4) >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        uint32_t run = 0u, done = 0u;  // tiles of all units so far, of this group
        WgItem w;
        while (next(w)) {
            const bool any = g == 0 || w.k1 >= 0;  // this group has a key tile
            const int kt = g ? w.k1 : w.k0, k = kt + row, cnt = w.qz - w.qa;
            float mul = p.qscale;
            if constexpr (Q8) {
                const int lp = k >> p.c.page_shift;
                const int page = any && k < w.hi && lp < p.max_pages ? __ldg(p.table + (long long)w.b * p.max_pages + lp) : -1;
                if (page >= 0 && page < p.c.num_pages) {
                    const int at = ((page * p.c.Hkv + w.h) << p.c.page_shift) + (k & ((1 << p.c.page_shift) - 1));
                    mul *= pow2f(min(max((int)__ldg(p.c.ke + at) - 127, -126), 127));
                }
            }
            // the tokens that see the key: [ia, iz)
            const int sink = p.window > 0 ? min(p.sinks, w.hi) : 0;
            const int ia = k - w.base;
            const int iz = p.window > 0 && k >= sink ? (int)min((long long)w.n, (long long)ia + p.window) : w.n;
            // whole tiles: all of their tokens see all keys
            const int first = kt + PG_TILE - 1 - w.base;
            const long long last = p.window > 0 && kt + PG_TILE > sink ? (long long)kt - w.base + p.window : w.n;
            float2 sum[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.0f, 0.0f);
            for (int j = 0; j < cnt; ++j) {
                const uint32_t at = run + (uint32_t)j;
                const int slot = 2 * g + (int)(done & 1u), ls = (int)(at % C::LST);
                const int it0 = w.i0 + (w.qa + j) * tqt;
                const bool whole = it0 >= first && it0 + tqt <= w.n && it0 + tqt <= last;
                const bool none = it0 + tqt <= kt - w.base;  // (all before the tile)
                uint32_t see[4] = {0u, 0u, 0u, 0u};
                if (!whole) {
                    const int lo = min(max(ia - it0, 0), 128) * p.GQ, hi = min(max(min(iz, w.n) - it0, 0), 128) * p.GQ;
#pragma unroll
                    for (int b = 0; b < 4; ++b) see[b] = ck_below(hi - 32 * b) & ~ck_below(lo - 32 * b);
                }
                if (any) await2(&bar.l_full[ls], (at / C::LST) & 1u, &bar.s_full[slot], (done >> 1) & 1u);
                else await(&bar.l_full[ls], (at / C::LST) & 1u);
                if (!ok) break;
                if (any) ++done;
                if (any && !none) {
                    qt_fence_after();
                    const float2 mul2 = make_float2(mul, mul);
                    const uint32_t ts = lanes + 128 * slot;
                    // 32 columns at a time, the next ones on their way from tensor memory
                    auto tile = [&](auto masked) {
                        constexpr bool MASKED = decltype(masked)::value;
                        uint32_t x[2][32];
                        qt_ld32(ts, x[0]);
                        qt_wait_ld();
                        qt_hold(x[0]);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (b < 3) qt_ld32(ts + 32 * (b + 1), x[(b + 1) & 1]);
                            const float4 *nl = reinterpret_cast<const float4 *>(slse + ls * 128 + 32 * b);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const uint32_t *y = x[b & 1] + c;
                                const float4 n4 = nl[c >> 2];
                                float2 t0 = __ffma2_rn(ck_f2(y[0], y[1]), mul2, make_float2(n4.x, n4.y));
                                float2 t1 = __ffma2_rn(ck_f2(y[2], y[3]), mul2, make_float2(n4.z, n4.w));
                                if constexpr (MASKED) {
                                    const uint32_t s = see[b] >> c;
                                    t0.x = s & 1u ? t0.x : NEG_INF;
                                    t0.y = s & 2u ? t0.y : NEG_INF;
                                    t1.x = s & 4u ? t1.x : NEG_INF;
                                    t1.y = s & 8u ? t1.y : NEG_INF;
                                }
                                float2 &s0 = sum[(c >> 1) & 2], &s1 = sum[((c >> 1) & 2) + 1];
                                s0 = __fadd2_rn(s0, make_float2(ex2(t0.x), ex2(t0.y)));
                                s1 = __fadd2_rn(s1, make_float2(ex2(t1.x), ex2(t1.y)));
                            }
                            if (b < 3) {
                                qt_wait_ld();
                                qt_hold(x[(b + 1) & 1]);
                            }
                            if (b == 2) {  // the last columns have come: the score tile's place is free
                                qt_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&bar.s_empty[slot]);
                            }
                        }
                    };
                    if (whole) tile(std::false_type());
                    else tile(std::true_type());
                } else if (any) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.s_empty[slot]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.l_empty[ls]);
            }
            if (!ok) break;
            run += (uint32_t)max(cnt, 0);
            if (any && k < p.keys)
                p.scores[(((size_t)w.b * p.Hkv + w.h) * p.srows + w.part) * p.keys + k] =
                    ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
        }
    } else if constexpr (Q8) {
        if (warp >= 12) {
            // -------------------------------------------- codes to operands
            const int j = threadIdx.x - 12 * 32;
            PgRing<C::RAW ? C::RAW : 1> raw;
            PgRing<C::KST> ks;
            WgItem w;
            while (next(w)) {
                if (w.qa >= w.qz) continue;
                for (int t = 0; t < (w.k1 < 0 ? 1 : 2); ++t) {
                    await(&bar.raw_full[raw.s], raw.par);
                    await(&bar.k_empty[ks.s], ks.par ^ 1u);
                    if (!ok) break;
                    // eight lanes a row; the upper four store their second half first, so
                    // that the eight fill all banks
                    const unsigned char *src = sraw + raw.s * RAW_B + swz128(j >> 3, j & 7);
                    unsigned char *dst = sk + ks.s * TILE_B + ((j & 7) >> 2) * HALF_B;
                    const bool odd = (j & 4) != 0;
                    const uint32_t d0 = swz128(j >> 3, 2 * (j & 3) + odd), d1 = swz128(j >> 3, 2 * (j & 3) + !odd);
#pragma unroll 2
                    for (int i = 0; i < PG_TILE / (4 * C::CONV); ++i) {
                        const int step = 128 * 4 * C::CONV * i;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + step);
                        uint4 x0, x1;
                        wg_operand<T>(odd ? v.z : v.x, x0.x, x0.y);
                        wg_operand<T>(odd ? v.w : v.y, x0.z, x0.w);
                        wg_operand<T>(odd ? v.x : v.z, x1.x, x1.y);
                        wg_operand<T>(odd ? v.y : v.w, x1.z, x1.w);
                        *reinterpret_cast<uint4 *>(dst + d0 + step) = x0;
                        *reinterpret_cast<uint4 *>(dst + d1 + step) = x1;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.raw_empty[raw.s]);
                        mbar_arrive(&bar.k_full[ks.s]);
                    }
                    raw.step();
                    ks.step();
                }
                if (!ok) break;
            }
        }
    }

    qt_fence_before();
    __syncthreads();
    qt_fence_after();
    if (warp == 1) tmem_free(tmem, 512);
}

template <class T, bool Q8> cudaError_t launch_weigh(const PagedAttendParams &p, cudaStream_t stream)
{
    auto kern = paged_weigh_kernel<T, Q8>;
    constexpr int smem = WgShape<Q8>::SMEM;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(p.large.G), WgShape<Q8>::THREADS, smem, stream, p);
}

// ------------------------------------------------------------- the update
//
// Each CTA takes an even share of the units (sequence, head, 8 tiles of keys) in
// their order; a thread has four keys, whose scores, rows' lse and weights it reads
// with all loads in flight, while it finds the next unit's.  Bound by memory: 4 bytes
// a row and key (of which most are still in L2) and 8 for the weight; 64 sequences of
// up to 16384 tokens, 8 kv heads of 4: 20 us, 107 MB.
constexpr int UPD_THREADS = 256, UPD_TILES = UPD_THREADS / 32;
constexpr int UPD_ROWS = 4;  // rows' scores in flight

__global__ void __launch_bounds__(UPD_THREADS, 4) paged_weigh_update_kernel(const __grid_constant__ PagedAttendParams p)
{
    __shared__ long long sums[UPD_THREADS / 32];
    __shared__ int at[3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto groups = [&](int b, PgEntry &e, int &start, int &n) -> int {
        int len = 0;
        (void)sequence(p, b, start, n, len);
        if (n == 0) return 0;
        e = make_entry(p, b, start, n, len, n, 0);
        return (e.ntiles + UPD_TILES - 1) / UPD_TILES;
    };
    PgEntry e;
    int start = 0, n = 0;
    const int per = (p.B + UPD_THREADS - 1) / UPD_THREADS, b0 = threadIdx.x * per, b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += (long long)groups(b, e, start, n) * p.Hkv;
    long long x = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, x, s);
        if (lane >= s) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < UPD_THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    Shares sh;
    sh.set(total, gridDim.x);
    if ((int)blockIdx.x >= sh.g) {
        pg_wait();
        return;
    }
    const long long u0 = sh.first(blockIdx.x);
    if (u0 >= before && u0 < before + mine) {  // one thread: the share starts in its sequences
        for (int b = b0; b < b1; ++b) {
            const int gs = groups(b, e, start, n);
            if (u0 < before + (long long)gs * p.Hkv) {
                const int r = (int)(u0 - before);
                at[0] = b;
                at[1] = r / gs;
                at[2] = r % gs;
                break;
            }
            before += (long long)gs * p.Hkv;
        }
    }
    __syncthreads();
    int b = at[0], h = at[1], g = at[2];
    int left = (int)(sh.first(blockIdx.x + 1) - u0), gs = groups(b, e, start, n);
    // Where this thread's four keys of a unit are: their weights (null: nothing to do),
    // scores or sums, and the rows of those.
    struct Four {
        float *w;
        const float *s;
        const float *l;  // the rows' lse (null: sums of a chunk's parts)
        int rows;
        uint32_t see;    // bits of the keys that are seen, and (from bit 4 on) that are new
    };
    auto find = [&]() {
        Four f;
        f.w = nullptr;
        PgView view;
        view.set(e, p.window, p.sinks);
        const int t = UPD_TILES * g + warp, k = pg_tile_key(e, t) + 4 * lane;
        if (t >= e.ntiles || !view.any(k, k + 4)) return f;
        const int lp = k >> p.c.page_shift;
        const int page = lp < p.max_pages ? __ldg(p.table + (long long)b * p.max_pages + lp) : -1;
        if (page < 0 || page >= p.c.num_pages) return f;
        f.w = p.weights + (((size_t)page * p.c.Hkv + h) << p.c.page_shift) + (k & ((1 << p.c.page_shift) - 1));
        const bool large = n * p.GQ > p.small_rows;
        const int r0 = large ? 0 : pg_counted(p, n) * p.GQ;
        f.rows = large ? pg_parts(p, n) : n * p.GQ - r0;
        f.s = p.scores + (((size_t)b * p.Hkv + h) * p.srows + r0) * p.keys + k;
        f.l = large ? nullptr : p.lse + ((size_t)h * p.T + start) * p.GQ + r0;
        f.see = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) f.see |= (view.one(k + i) ? 1u << i : 0u) | (k + i >= e.p0 ? 16u << i : 0u);
        return f;
    };
    auto step = [&]() -> bool {  // to the share's next unit
        if (--left <= 0) return false;
        if (++g == gs) {
            g = 0;
            if (++h == p.Hkv) {
                h = 0;
                do gs = ++b < p.B ? groups(b, e, start, n) : 1;
                while (gs == 0);
            }
        }
        return true;
    };
    Four f = find();
    pg_wait();  // (for the scores and sums; the shares come of the call's inputs)
    for (bool more = true; more;) {
        const Four now = f;
        float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f), s[UPD_ROWS];
        float l[UPD_ROWS];
        auto fetch = [&](int r) {
#pragma unroll
            for (int i = 0; i < UPD_ROWS; ++i) {
                if (r + i >= now.rows) break;
                s[i] = __ldcs(reinterpret_cast<const float4 *>(now.s + (size_t)(r + i) * p.keys));
                l[i] = now.l ? now.l[r + i] : 0.0f;
            }
        };
        if (now.w) {
            old = *reinterpret_cast<const float4 *>(now.w);
            fetch(0);
        }
        more = step();
        if (more) f = find();  // (the next unit's page, while this one's numbers come)
        if (!now.w) continue;
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r = 0;;) {
#pragma unroll
            for (int i = 0; i < UPD_ROWS; ++i) {
                if (r + i >= now.rows) break;
                a[0] += now.l ? ex2(s[i].x - l[i]) : s[i].x;
                a[1] += now.l ? ex2(s[i].y - l[i]) : s[i].y;
                a[2] += now.l ? ex2(s[i].z - l[i]) : s[i].z;
                a[3] += now.l ? ex2(s[i].w - l[i]) : s[i].w;
            }
            r += UPD_ROWS;
            if (r >= now.rows) break;
            fetch(r);
        }
        // (decay 0 does not ask what was there)
        auto sum = [&](int i, float o) {
            return ((now.see >> (4 + i)) & 1u) || p.decay == 0.0f ? a[i] : fmaf(p.decay, o, a[i]);
        };
        const float4 y = make_float4(sum(0, old.x), sum(1, old.y), sum(2, old.z), sum(3, old.w));
        if ((now.see & 15u) == 15u) {
            *reinterpret_cast<float4 *>(now.w) = y;
        } else {
            if (now.see & 1u) now.w[0] = y.x;
            if (now.see & 2u) now.w[1] = y.y;
            if (now.see & 4u) now.w[2] = y.z;
            if (now.see & 8u) now.w[3] = y.w;
        }
    }
}

}  // namespace

cudaError_t launch_paged_weigh(const PagedAttendParams &p0, int q_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAttendParams p = p0;
    const bool q8 = cache_dtype == VQ_E4M3;
    const uint64_t rows = ((uint64_t)p.c.num_pages * p.c.Hkv) << p.c.page_shift;
    const uint32_t box = 1u << p.c.page_shift < (unsigned)PG_TILE ? 1u << p.c.page_shift : (unsigned)PG_TILE;
    if (!encode_tmap_pages(&p.tmk, p.c.k, rows, q8 ? 1 : 2, box) || !encode_tmap_queries(&p.tmq, p)) return cudaErrorInvalidValue;
    if (q_dtype == VQ_F16) return q8 ? launch_weigh<__half, true>(p, stream) : launch_weigh<__half, false>(p, stream);
    return q8 ? launch_weigh<__nv_bfloat16, true>(p, stream) : launch_weigh<__nv_bfloat16, false>(p, stream);
}

cudaError_t launch_paged_weigh_update(const PagedAttendParams &p, cudaStream_t stream)
{
    const int G = p.small.cap ? p.small.G : p.large.G;
    return launch_early(paged_weigh_update_kernel, dim3(4 * G), UPD_THREADS, 0, stream, p);
}

cudaError_t paged_weigh_take_device_error(unsigned *bits, cudaStream_t stream)
{
    *bits = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_pw_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (*bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_pw_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace vq
