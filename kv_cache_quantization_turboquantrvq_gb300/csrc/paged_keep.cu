// paged_keep.cu - keeping a part of a paged key/value cache (sm_103a): the choice
// of the tokens that stay by their accumulated softmax weights, and moving the
// tokens that stay together.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pe_err);

namespace cg = cooperative_groups;

// --------------------------------------------------------------- the choice
//
// Of a sequence of L > budget tokens each kv head keeps the first `sinks`, the
// last `recent`, and of the middle the `need` = budget - sinks - recent of largest
// weight, of equal weights the earlier ones; ascending.
//
// The need-th largest weight is found digit by digit (11, 11 and 10 bits from the
// top) on numbers whose order as integers is the weights' order: a histogram of
// the digit over the weights that share the digits before it, then the digit at
// which the counts from above reach `need`.  What lies above is taken, what shares
// all digits is taken in the tokens' order while it is needed.  The first
// histogram is made while the weights are read; they stay in shared memory for
// the other passes, so each is read once.
//
// A cluster of CTAs takes one row (sequence, head), each CTA a contiguous part of
// it; they read one another's histograms and counts.  Weights are handled four
// tokens at a time (a page holds whole fours), those of tokens outside the middle
// as 0, which no weight is.
//
// 2048 of up to 16384 tokens, 512 rows: 27 us, where reading the weights takes 3; 8192
// of 131072, 8 rows in clusters of 8: 23 us.  A block's chain (page, weights, three
// digits with a scan each, counts, list) bounds it: token by token it took 48 us,
// with 256 threads and two blocks a row 35.
constexpr int SEL_THREADS = 512, SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_BINS = 2048;
constexpr int SEL_MAX = 10240, SEL_PAIR = 6000;  // fours of a CTA that stay in shared memory: of one on an SM, of two
constexpr int SEL_OWN = SEL_BINS / SEL_THREADS;  // bins of a thread
static_assert(SEL_OWN * SEL_THREADS == SEL_BINS && SEL_OWN % 4 == 0, "whole fours of bins a thread");

struct SelShared {
    unsigned hist[2][SEL_BINS];
    unsigned warp_sum[SEL_WARPS], warp_gt[SEL_WARPS], warp_tie[SEL_WARPS];
    unsigned gt, tie;                // of this CTA's part
    unsigned bin, above, inside;     // the digit's bin, what lies above it, what lies in it
};

// The order of weights as integers, none of them 0: 0 and -0 alike, NaN largest.
__device__ __forceinline__ unsigned sel_key(float x)
{
    if (x != x) return 0xffffffffu;
    const unsigned u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(SEL_THREADS, 2) paged_select_kernel(const __grid_constant__ PagedSelectParams p)
{
    extern __shared__ __align__(16) unsigned char sel_raw[];
    SelShared &s = *reinterpret_cast<SelShared *>(sel_raw);
    static_assert(sizeof(SelShared) % 4 == 0, "fours behind it");
    uint4 *keys = reinterpret_cast<uint4 *>(sel_raw + (sizeof(SelShared) + 15) / 16 * 16);  // [p.held]
    const cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)blockIdx.x / cs, b = row / p.Hkv, h = row - b * p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = (int)((long long)p.max_pages << p.page_shift);
    const int given = __ldg(p.lens + b), L = min(max(given, 0), cap);
    int32_t *keep = p.keep + (size_t)row * p.budget;
    if (rank == 0 && tid == 0) {
        if (given != L && h == 0) atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        if (h == 0) p.counts[b] = min(L, p.budget);
    }
    const int all = cs * SEL_THREADS, me = rank * SEL_THREADS + tid;
    if (L <= p.budget) {  // (the whole cluster)
        for (int i = me; i < p.budget; i += all) keep[i] = i < L ? i : -1;
        return;
    }
    for (int i = me; i < p.sinks; i += all) keep[i] = i;
    for (int i = me; i < p.recent; i += all) keep[p.budget - p.recent + i] = L - p.recent + i;
    const int m0 = p.sinks, m1 = L - p.recent;  // the middle
    int need = p.budget - p.sinks - p.recent;
    if (need == 0) return;
    auto together = [&] {  // a barrier of the cluster
        if (cs == 1) __syncthreads();
        else cluster.sync();
    };

    const int fours = (m1 + 3) / 4 - m0 / 4, seg = (fours + cs - 1) / cs, s0 = min(rank * seg, fours);
    const int n = min(seg, fours - s0), t0 = 4 * (m0 / 4 + s0);  // this CTA's fours, and its first token
    const int32_t *table = p.table + (size_t)b * p.max_pages;
    const int in_page = (1 << p.page_shift) - 1;
    auto keys_of = [&](int t, float4 x) {
        uint4 k = make_uint4(sel_key(x.x), sel_key(x.y), sel_key(x.z), sel_key(x.w));
        if (t < m0 || t + 4 > m1) {
            k.x = t >= m0 && t < m1 ? k.x : 0u;
            k.y = t + 1 >= m0 && t + 1 < m1 ? k.y : 0u;
            k.z = t + 2 >= m0 && t + 2 < m1 ? k.z : 0u;
            k.w = t + 3 >= m0 && t + 3 < m1 ? k.w : 0u;
        }
        return k;
    };
    // the weights of tokens t .. t + 3, which lie in this page; the lowest: it is not in the pool
    auto weights_of = [&](int t, int page) {
        const float low = -__builtin_huge_valf();
        if ((unsigned)page >= (unsigned)p.num_pages) return make_float4(low, low, low, low);
        return __ldg(reinterpret_cast<const float4 *>(p.weights + ((((size_t)page * p.Hkv + h) << p.page_shift) + (t & in_page))));
    };
    auto four = [&](int i) -> uint4 {
        if (i < p.held) return keys[i];
        const int t = t0 + 4 * i;
        return keys_of(t, weights_of(t, __ldg(table + (t >> p.page_shift))));
    };

    for (int i = tid; i < SEL_BINS; i += SEL_THREADS) s.hist[0][i] = 0u;
    __syncthreads();
    constexpr int U = 4;
    for (int i0 = tid; i0 < n; i0 += U * SEL_THREADS) {
        int page[U];
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) page[u] = __ldg(table + ((t0 + 4 * min(i0 + u * SEL_THREADS, n - 1)) >> p.page_shift));
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = weights_of(t0 + 4 * min(i0 + u * SEL_THREADS, n - 1), page[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * SEL_THREADS;
            if (i >= n) break;
            const uint4 k = keys_of(t0 + 4 * i, x[u]);
            if (i < p.held) keys[i] = k;
            if ((unsigned)page[u] >= (unsigned)p.num_pages) atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
            if (k.x) atomicAdd(&s.hist[0][k.x >> 21], 1u);
            if (k.y) atomicAdd(&s.hist[0][k.y >> 21], 1u);
            if (k.z) atomicAdd(&s.hist[0][k.z >> 21], 1u);
            if (k.w) atomicAdd(&s.hist[0][k.w >> 21], 1u);
        }
    }
    unsigned lo = 0u, hi = 0xffffffffu;  // weights above hi are taken, of [lo, hi] the first `need`
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int buf = pass & 1;
        if (pass > 0) {
            auto count = [&](unsigned k) {
                if (k - lo <= hi - lo) atomicAdd(&s.hist[buf][(k - lo) >> shift], 1u);
            };
            for (int i = tid; i < n; i += SEL_THREADS) {
                const uint4 k = four(i);
                count(k.x);
                count(k.y);
                count(k.z);
                count(k.w);
            }
        }
        together();
        // a thread's bins, from the top
        const int b0 = SEL_BINS - SEL_OWN * (tid + 1);
        unsigned c[SEL_OWN];
#pragma unroll
        for (int i = 0; i < SEL_OWN; ++i) c[i] = 0u;
        for (int r = 0; r < cs; ++r) {
            const unsigned *other = cs == 1 ? s.hist[buf] : cluster.map_shared_rank(s.hist[buf], r);
#pragma unroll
            for (int i = 0; i < SEL_OWN; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(other + b0 + i);
                c[i] += x.x; c[i + 1] += x.y; c[i + 2] += x.z; c[i + 3] += x.w;
            }
        }
        // (the other buffer's readers have passed the barrier above)
        for (int i = tid; i < SEL_BINS / 4; i += SEL_THREADS) reinterpret_cast<uint4 *>(s.hist[buf ^ 1])[i] = make_uint4(0u, 0u, 0u, 0u);
        unsigned sum = 0u;
#pragma unroll
        for (int i = 0; i < SEL_OWN; ++i) sum += c[i];
        unsigned x = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(FULL_MASK, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s.warp_sum[warp] = x;
        __syncthreads();
        unsigned above = x - sum + __reduce_add_sync(FULL_MASK, lane < warp ? s.warp_sum[lane] : 0u);
        if (above < (unsigned)need && above + sum >= (unsigned)need) {  // one thread
            bool found = false;
#pragma unroll
            for (int i = SEL_OWN - 1; i >= 0; --i) {
                if (!found && above + c[i] >= (unsigned)need) {
                    found = true;
                    s.bin = (unsigned)(b0 + i);
                    s.above = above;
                    s.inside = c[i];
                }
                above += c[i];
            }
        }
        __syncthreads();
        need -= (int)s.above;
        const unsigned from = lo + (s.bin << shift);
        hi = min(hi, from + ((1u << shift) - 1u));
        lo = max(from, 1u);  // (not the tokens outside the middle)
        const bool done = s.inside == (unsigned)need;
        __syncthreads();
        if (done) break;
    }

    // taken tokens of this CTA's part, warp by warp, then of all parts before
    const int per = ((n + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
    const int w0 = min(warp * per, n), w1 = min(w0 + per, n);
    auto over = [&](unsigned k) { return k > hi ? 1u : 0u; };
    auto even = [&](unsigned k) { return k - lo <= hi - lo ? 1u : 0u; };
    unsigned gt = 0u, tie = 0u;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint4 k = four(i);
        gt += over(k.x) + over(k.y) + over(k.z) + over(k.w);
        tie += even(k.x) + even(k.y) + even(k.z) + even(k.w);
    }
    gt = __reduce_add_sync(FULL_MASK, gt);
    tie = __reduce_add_sync(FULL_MASK, tie);
    if (lane == 0) {
        s.warp_gt[warp] = gt;
        s.warp_tie[warp] = tie;
    }
    __syncthreads();
    unsigned bg = 0u, bt = 0u;
    if (cs > 1) {
        if (tid == 0) {
            unsigned g = 0u, t = 0u;
            for (int w = 0; w < SEL_WARPS; ++w) {
                g += s.warp_gt[w];
                t += s.warp_tie[w];
            }
            s.gt = g;
            s.tie = t;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            bg += *cluster.map_shared_rank(&s.gt, r);
            bt += *cluster.map_shared_rank(&s.tie, r);
        }
    }
    bg += __reduce_add_sync(FULL_MASK, lane < warp ? s.warp_gt[lane] : 0u);
    bt += __reduce_add_sync(FULL_MASK, lane < warp ? s.warp_tie[lane] : 0u);
    int32_t *dst = keep + p.sinks;
    for (int i = w0; i < w1; i += 32) {
        const uint4 k = i + lane < w1 ? four(i + lane) : make_uint4(0u, 0u, 0u, 0u);
        // counts of both kinds in one number: at most 128 of each
        const unsigned mine = (over(k.x) + over(k.y) + over(k.z) + over(k.w)) << 16 | (even(k.x) + even(k.y) + even(k.z) + even(k.w));
        unsigned x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(FULL_MASK, x, d);
            if (lane >= d) x += y;
        }
        unsigned g = bg + ((x - mine) >> 16), t = bt + ((x - mine) & 0xffffu);
        auto put = [&](unsigned kk, int j) {
            const bool eq = even(kk) != 0u;
            if (over(kk) || (eq && t < (unsigned)need)) dst[g + min(t, (unsigned)need)] = t0 + 4 * (i + lane) + j;
            g += over(kk);
            t += eq ? 1u : 0u;
        };
        if (mine) {
            put(k.x, 0);
            put(k.y, 1);
            put(k.z, 2);
            put(k.w, 3);
        }
        const unsigned total = __shfl_sync(FULL_MASK, x, 31);
        bg += total >> 16;
        bt += total & 0xffffu;
    }
    if (cs > 1) cluster.sync();  // (the counts are read by others)
}

// ------------------------------------------------------------- moving rows
//
// Token keep[b][h][i] goes to place first[b] + i of its sequence, which is never
// behind it, in place.  A cluster takes one row (sequence, head) in rounds of
// MOVE_ROWS tokens a CTA: all tokens of a round are read before any is written,
// and the places that a round writes lie before every token that a later round
// reads - so the next rounds' tokens are already on their way (asynchronous copies
// to shared memory, where the lane that asked for them takes them) while this
// round waits for the cluster and writes.  A row's list entry, its pages and its
// data come one after another, each a round ahead of its use (all in the round of
// the copy: 4096 tokens of 16 x 8 rows 177 us; without copies ahead 138).
//
// 4096 tokens of 16 x 8 rows, bf16: 114 us, 4.8 TB/s.  The rounds and their barrier
// bound it: the same rows copied from and to the same kind of places, but in another
// pool and each for itself, take 84 us (6.4 TB/s).
constexpr int MOVE_THREADS = 256, MOVE_R = 4, MOVE_ROWS = MOVE_THREADS / 16 * MOVE_R, MOVE_STAGES = 3;
constexpr int MOVE_AHEAD = MOVE_STAGES - 1;  // rounds that are copied ahead
constexpr int MOVE_SLOTS = 8;                // rounds whose rows are known

template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

template <class V>  // what each of 16 lanes moves of a row: uint4 of 16-bit entries, uint2 of codes
__global__ void __launch_bounds__(MOVE_THREADS) paged_compact_kernel(const __grid_constant__ PagedCompactParams p)
{
    constexpr bool Q8 = sizeof(V) == 8;
    extern __shared__ __align__(16) unsigned char move_raw[];
    __shared__ int2 s_rows[MOVE_SLOTS][MOVE_ROWS];  // of the pool: from, to; to -1: the row stays, or is left out
    V *buf = reinterpret_cast<V *>(move_raw) + threadIdx.x;  // [stage][row of the lane][key, value], THREADS apart
    const cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)blockIdx.x / cs, b = row / p.c.Hkv, h = row - b * p.c.Hkv;
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int cap = (int)((long long)p.max_pages << p.c.page_shift);
    const int32_t *keep = p.keep + b * p.keep_b + h * p.keep_h, *table = p.table + (size_t)b * p.max_pages;
    const int given = __ldg(p.counts + b), at = p.first ? __ldg(p.first + b) : 0;
    int n = min(max(given, 0), p.K);
    const bool inside = at >= 0 && at <= cap;
    if (!inside) n = 0;
    if ((given != n || !inside) && threadIdx.x == 0) atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
    const int step = cs * MOVE_ROWS, rounds = (n + step - 1) / step;
    // The first threads find a row each, in three steps: its list entry (and the one
    // before), the pages of both ends, its rows of the pool.
    struct Entry { int t, before; };
    struct Ends { int t, from, to; };  // t < 0: nothing to move
    const int i0 = rank * MOVE_ROWS + (int)threadIdx.x;  // (of the first round)
    auto entry = [&](int round) {
        const int i = round * step + i0;
        Entry e = {-1, -1};
        if (round < rounds && i < n) {
            e.t = __ldg(keep + i);
            e.before = i > 0 ? __ldg(keep + i - 1) : -1;
        }
        return e;
    };
    auto ends = [&](int round, Entry e) {
        const int i = round * step + i0;
        Ends x = {-1, -1, -1};
        if (round >= rounds || i >= n) return x;
        if (e.t <= e.before || e.t < at + i || e.t >= cap) {
            atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        } else if (e.t > at + i) {  // (else it stays where it is)
            x.t = e.t;
            x.from = __ldg(table + (e.t >> p.c.page_shift));
            x.to = __ldg(table + ((at + i) >> p.c.page_shift));
        }
        return x;
    };
    auto rows = [&](int round, Ends x) {
        int2 r = make_int2(-1, -1);
        if (x.t >= 0) {
            const int in = (1 << p.c.page_shift) - 1;
            if (x.from >= 0 && x.from < p.c.num_pages && x.to >= 0 && x.to < p.c.num_pages)
                r = make_int2(((x.from * p.c.Hkv + h) << p.c.page_shift) + (x.t & in),
                              ((x.to * p.c.Hkv + h) << p.c.page_shift) + ((at + round * step + i0) & in));
            else
                atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        }
        s_rows[round % MOVE_SLOTS][threadIdx.x] = r;
    };
    const bool finds = threadIdx.x < MOVE_ROWS;
    Entry e = {-1, -1};
    Ends x = {-1, -1, -1};
    if (finds) {
        Entry e3[MOVE_STAGES];
        Ends x3[MOVE_STAGES];
#pragma unroll
        for (int s = 0; s < MOVE_STAGES; ++s) e3[s] = entry(s);
        const Entry e4 = entry(MOVE_STAGES);
        e = entry(MOVE_STAGES + 1);
#pragma unroll
        for (int s = 0; s < MOVE_STAGES; ++s) x3[s] = ends(s, e3[s]);
        x = ends(MOVE_STAGES, e4);
#pragma unroll
        for (int s = 0; s < MOVE_STAGES; ++s) rows(s, x3[s]);
    }
    __syncthreads();
    uint32_t part[MOVE_STAGES][MOVE_R] = {};  // a row's exponents and weight, a lane each
    auto fetch = [&](int round, uint32_t (&small)[MOVE_R], int stage) {
#pragma unroll
        for (int j = 0; j < MOVE_R; ++j) {
            const int2 r = s_rows[round % MOVE_SLOTS][j * (MOVE_THREADS / 16) + group];
            if (r.y < 0) continue;
            V *d = buf + (stage * MOVE_R + j) * 2 * MOVE_THREADS;
            copy_async<sizeof(V)>(d, static_cast<const V *>(p.c.k) + (size_t)r.x * 16 + lane);
            copy_async<sizeof(V)>(d + MOVE_THREADS, static_cast<const V *>(p.c.v) + (size_t)r.x * 16 + lane);
            if (Q8 && lane < 2) small[j] = (lane ? p.c.ve : p.c.ke)[r.x];
            if (p.weights && lane == 2) small[j] = __float_as_uint(p.weights[r.x]);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < MOVE_AHEAD; ++s) fetch(s, part[s], s);
    for (int r0 = 0; r0 < rounds; r0 += MOVE_STAGES) {
#pragma unroll
        for (int s = 0; s < MOVE_STAGES; ++s) {
            const int r = r0 + s;
            if (r >= rounds) break;
            fetch(r + MOVE_AHEAD, part[(s + MOVE_AHEAD) % MOVE_STAGES], (s + MOVE_AHEAD) % MOVE_STAGES);
            // (rows of the round after that one, which the barrier below shows to all)
            if (finds) {
                rows(r + MOVE_STAGES, x);
                x = ends(r + MOVE_STAGES + 1, e);
                e = entry(r + MOVE_STAGES + 2);
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(MOVE_AHEAD) : "memory");  // this round's rows are here
            // and the small parts of them: a number made of them is there when they are
            bool odd = false;
#pragma unroll
            for (int j = 0; j < MOVE_R; ++j) odd ^= (part[s][j] & 1u) != 0u;
            __syncthreads_or(odd);
            // All that the cluster's barrier has to order are these reads, which are done;
            // with a fence it would wait for the writes of the round before.
            if (cs > 1) {
                asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
                asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
            }
#pragma unroll
            for (int j = 0; j < MOVE_R; ++j) {
                const int to = s_rows[r % MOVE_SLOTS][j * (MOVE_THREADS / 16) + group].y;
                if (to < 0) continue;
                const V *d = buf + (s * MOVE_R + j) * 2 * MOVE_THREADS;
                static_cast<V *>(const_cast<void *>(p.c.k))[(size_t)to * 16 + lane] = d[0];
                static_cast<V *>(const_cast<void *>(p.c.v))[(size_t)to * 16 + lane] = d[MOVE_THREADS];
                if (Q8 && lane < 2) const_cast<uint8_t *>(lane ? p.c.ve : p.c.ke)[to] = (uint8_t)part[s][j];
                if (p.weights && lane == 2) p.weights[to] = __uint_as_float(part[s][j]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class... A, class... B>
cudaError_t launch_clusters(void (*kern)(A...), unsigned rows, int cs, int threads, size_t smem, cudaStream_t stream, const B &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * (unsigned)cs);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectParams &p0, cudaStream_t stream)
{
    PagedSelectParams p = p0;
    const unsigned rows = (unsigned)p.B * (unsigned)p.Hkv;
    const long long cap = (long long)p.max_pages << p.page_shift;
    // CTAs a row: more than one where there are few rows (8 rows of 131072 tokens with 1,
    // 2, 4 and 8: 132, 65, 26 and 22 us; 512 rows of up to 16384: 29, 39, 72 and 230;
    // each over several pools in turn).  Not by the block table's width, which says
    // little about the lengths: those 512 rows in a table for 131072 take 29 us with
    // one and 71 with the four that could keep all of that (512 rows that do have 131072
    // tokens 389 with one, 303 with two).
    int cs = 1;
    while (cs < 8 && cap / cs > SEL_BINS && (long long)rows * cs < sm_count()) cs *= 2;
    // what is kept at hand leaves room for two CTAs an SM where there are many rows (the
    // wide table 36 us with SEL_MAX, 29 so; 512 rows of 131072 tokens 485 and 389)
    const long long most = (long long)rows * cs > 2 * sm_count() ? SEL_PAIR : SEL_MAX, held = (cap / 4 + 1 + cs) / cs;
    p.held = (int)(held < most ? held : most);
    constexpr size_t fixed = (sizeof(SelShared) + 15) / 16 * 16;
    const size_t smem = fixed + sizeof(uint4) * (size_t)p.held;
    cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(fixed + sizeof(uint4) * SEL_MAX));
    if (e != cudaSuccess) return e;
    return launch_clusters(paged_select_kernel, rows, cs, SEL_THREADS, smem, stream, p);
}

cudaError_t launch_paged_compact(const PagedCompactParams &p, int cache_dtype, cudaStream_t stream)
{
    const unsigned rows = (unsigned)p.B * (unsigned)p.c.Hkv;
    const int chunks = (p.K + MOVE_ROWS - 1) / MOVE_ROWS;
    // CTAs a row: as many as fill the SMs twice (4096 tokens of 8 rows with 1, 2, 4 and
    // 8: 107, 60, 33 and 21 us; of 128 rows 134, 113, 115 and 120)
    int cs = 1;
    while (cs < 8 && cs < chunks && (long long)rows * cs < 2 * sm_count()) cs *= 2;
    const bool q8 = cache_dtype == VQ_E4M3;
    const int smem = MOVE_STAGES * MOVE_R * 2 * MOVE_THREADS * (q8 ? (int)sizeof(uint2) : (int)sizeof(uint4));
    auto kern = q8 ? paged_compact_kernel<uint2> : paged_compact_kernel<uint4>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_clusters(kern, rows, cs, MOVE_THREADS, smem, stream, p);
}

cudaError_t paged_keep_take_device_error(unsigned *bits, cudaStream_t stream)
{
    *bits = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_pe_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (*bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_pe_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace vq
