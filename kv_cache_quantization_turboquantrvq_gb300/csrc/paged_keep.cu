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
// it; they read one another's histograms and counts.
constexpr int SEL_THREADS = 512, SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_BINS = 2048;
constexpr int SEL_MAX = 40960;  // weights of a CTA that stay in shared memory
static_assert(SEL_BINS == 4 * SEL_THREADS, "four bins a thread");

struct SelShared {
    unsigned hist[2][SEL_BINS];
    unsigned warp_sum[SEL_WARPS], warp_gt[SEL_WARPS], warp_tie[SEL_WARPS];
    unsigned gt, tie;                // of this CTA's part
    unsigned bin, above, inside;     // the digit's bin, what lies above it, what lies in it
};

// The order of weights as integers: 0 and -0 alike, NaN largest.
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
    unsigned *keys = reinterpret_cast<unsigned *>(sel_raw + sizeof(SelShared));  // [p.held]
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
    const int mid = L - p.sinks - p.recent;
    int need = p.budget - p.sinks - p.recent;
    if (need == 0) return;

    const int seg = (mid + cs - 1) / cs, s0 = min(rank * seg, mid), n = min(seg, mid - s0);  // this CTA's part
    const int t0 = p.sinks + s0;                                                             // its first token
    const int32_t *table = p.table + (size_t)b * p.max_pages;
    auto fetch = [&](int i) -> unsigned {  // of token t0 + i
        const int t = t0 + i, page = __ldg(table + (t >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
            atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
            return 0u;
        }
        return sel_key(__ldg(p.weights + (((size_t)page * p.Hkv + h) << p.page_shift) + (t & ((1 << p.page_shift) - 1))));
    };
    auto key = [&](int i) { return i < p.held ? keys[i] : fetch(i); };

    for (int i = tid; i < SEL_BINS; i += SEL_THREADS) s.hist[0][i] = 0u;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += 8 * SEL_THREADS) {
        unsigned k[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * SEL_THREADS + tid;
            k[u] = i < n ? fetch(i) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * SEL_THREADS + tid;
            if (i >= n) break;
            if (i < p.held) keys[i] = k[u];
            atomicAdd(&s.hist[0][k[u] >> 21], 1u);
        }
    }
    unsigned lo = 0u, hi = 0xffffffffu;  // weights above hi are taken, of [lo, hi] the first `need`
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int buf = pass & 1;
        if (pass > 0) {
            for (int i = tid; i < n; i += SEL_THREADS) {
                const unsigned k = key(i);
                if (k >= lo && k <= hi) atomicAdd(&s.hist[buf][(k - lo) >> shift], 1u);
            }
        }
        cluster.sync();
        // four bins a thread, from the top: bins 2044 - 4 tid ...
        const int b0 = SEL_BINS - 4 - 4 * tid;
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        for (int r = 0; r < cs; ++r) {
            const unsigned *other = cluster.map_shared_rank(s.hist[buf], r);
            const uint4 x = *reinterpret_cast<const uint4 *>(other + b0);
            c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
        }
        // (the other buffer's readers have passed the barrier above)
        for (int i = tid; i < SEL_BINS; i += SEL_THREADS) s.hist[buf ^ 1][i] = 0u;
        const unsigned four = c.x + c.y + c.z + c.w;
        unsigned x = four;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(FULL_MASK, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s.warp_sum[warp] = x;
        __syncthreads();
        unsigned above = x - four;
        for (int w = 0; w < warp; ++w) above += s.warp_sum[w];
        if (above < (unsigned)need && above + four >= (unsigned)need) {  // one thread
            const unsigned cc[4] = {c.w, c.z, c.y, c.x};
            int i = 0;
            while (above + cc[i] < (unsigned)need) above += cc[i++];
            s.bin = (unsigned)(b0 + 3 - i);
            s.above = above;
            s.inside = cc[i];
        }
        __syncthreads();
        need -= (int)s.above;
        lo += s.bin << shift;
        hi = lo + ((1u << shift) - 1u);
        const bool done = s.inside == (unsigned)need;
        __syncthreads();
        if (done) break;
    }

    // taken tokens of this CTA's part, warp by warp, then of all parts before
    const int per = ((n + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
    const int w0 = min(warp * per, n), w1 = min(w0 + per, n);
    unsigned gt = 0u, tie = 0u;
    for (int i = w0; i < w1; i += 32) {
        const unsigned k = i + lane < w1 ? key(i + lane) : 0u;
        const bool in = i + lane < w1;
        gt += __popc(__ballot_sync(FULL_MASK, in && k > hi));
        tie += __popc(__ballot_sync(FULL_MASK, in && k >= lo && k <= hi));
    }
    if (lane == 0) {
        s.warp_gt[warp] = gt;
        s.warp_tie[warp] = tie;
    }
    __syncthreads();
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
    unsigned bg = 0u, bt = 0u;
    for (int r = 0; r < rank; ++r) {
        bg += *cluster.map_shared_rank(&s.gt, r);
        bt += *cluster.map_shared_rank(&s.tie, r);
    }
    for (int w = 0; w < warp; ++w) {
        bg += s.warp_gt[w];
        bt += s.warp_tie[w];
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i = w0; i < w1; i += 32) {
        const bool in = i + lane < w1;
        const unsigned k = in ? key(i + lane) : 0u;
        const bool over = in && k > hi, eq = in && k >= lo && k <= hi;
        const unsigned mg = __ballot_sync(FULL_MASK, over), mt = __ballot_sync(FULL_MASK, eq);
        const unsigned ties = bt + __popc(mt & below);
        if (over || (eq && ties < (unsigned)need))
            keep[p.sinks + bg + __popc(mg & below) + min(ties, (unsigned)need)] = t0 + i + lane;
        bg += __popc(mg);
        bt += __popc(mt);
    }
    cluster.sync();  // (the counts are read by others)
}

// ------------------------------------------------------------- moving rows
//
// Token keep[b][h][i] goes to place first[b] + i of its sequence, which is never
// behind it, in place.  A cluster takes one row (sequence, head) in rounds of
// MOVE_ROWS tokens a CTA: all tokens of a round are read before any is written,
// and the places that a round writes lie before every token that a later round
// reads.
constexpr int MOVE_THREADS = 512, MOVE_R = 4, MOVE_ROWS = MOVE_THREADS / 16 * MOVE_R;

template <class V>  // what each of 16 lanes moves of a row: uint4 of 16-bit entries, uint2 of codes
__global__ void __launch_bounds__(MOVE_THREADS) paged_compact_kernel(const __grid_constant__ PagedCompactParams p)
{
    constexpr bool Q8 = sizeof(V) == 8;
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
    auto place = [&](int t) -> long long {  // row of the pool, -1: no such page
        const int page = __ldg(table + (t >> p.c.page_shift));
        if (page < 0 || page >= p.c.num_pages) return -1;
        return (((long long)page * p.c.Hkv + h) << p.c.page_shift) + (t & ((1 << p.c.page_shift) - 1));
    };
    for (int r0 = 0; r0 < n; r0 += cs * MOVE_ROWS) {
        V k[MOVE_R], v[MOVE_R];
        float w[MOVE_R];
        uint8_t ke[MOVE_R], ve[MOVE_R];
        long long src[MOVE_R], dst[MOVE_R];
#pragma unroll
        for (int j = 0; j < MOVE_R; ++j) {
            const int i = r0 + rank * MOVE_ROWS + j * (MOVE_THREADS / 16) + group;
            src[j] = -1;
            if (i >= n) continue;
            const int t = __ldg(keep + i), before = i > 0 ? __ldg(keep + i - 1) : -1;
            if (t == at + i && t < cap) continue;  // stays where it is
            if (t > before && t > at + i && t < cap) {
                src[j] = place(t);
                dst[j] = place(at + i);
                if (dst[j] < 0) src[j] = -1;
            }
            if (src[j] < 0 && lane == 0) atomicOr(&g_pe_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        }
#pragma unroll
        for (int j = 0; j < MOVE_R; ++j) {
            if (src[j] < 0) continue;
            k[j] = __ldcs(static_cast<const V *>(p.c.k) + src[j] * 16 + lane);
            v[j] = __ldcs(static_cast<const V *>(p.c.v) + src[j] * 16 + lane);
            if (lane == 0) {
                if constexpr (Q8) {
                    ke[j] = p.c.ke[src[j]];
                    ve[j] = p.c.ve[src[j]];
                }
                if (p.weights) w[j] = p.weights[src[j]];
            }
        }
        cluster.sync();
#pragma unroll
        for (int j = 0; j < MOVE_R; ++j) {
            if (src[j] < 0) continue;
            static_cast<V *>(const_cast<void *>(p.c.k))[dst[j] * 16 + lane] = k[j];
            static_cast<V *>(const_cast<void *>(p.c.v))[dst[j] * 16 + lane] = v[j];
            if (lane == 0) {
                if constexpr (Q8) {
                    const_cast<uint8_t *>(p.c.ke)[dst[j]] = ke[j];
                    const_cast<uint8_t *>(p.c.ve)[dst[j]] = ve[j];
                }
                if (p.weights) p.weights[dst[j]] = w[j];
            }
        }
    }
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
    int cs = 1;
    while (cs < 8 && cap / cs > SEL_BINS && ((long long)rows * cs < sm_count() || cap / cs > SEL_MAX)) cs *= 2;
    p.held = (int)(cap / cs + 1 < SEL_MAX ? cap / cs + 1 : SEL_MAX);
    const size_t smem = sizeof(SelShared) + sizeof(unsigned) * (size_t)p.held;
    cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(SelShared) + sizeof(unsigned) * SEL_MAX));
    if (e != cudaSuccess) return e;
    return launch_clusters(paged_select_kernel, rows, cs, SEL_THREADS, smem, stream, p);
}

cudaError_t launch_paged_compact(const PagedCompactParams &p, int cache_dtype, cudaStream_t stream)
{
    const unsigned rows = (unsigned)p.B * (unsigned)p.c.Hkv;
    const int chunks = (p.K + MOVE_ROWS - 1) / MOVE_ROWS;
    int cs = 1;
    while (cs < 8 && cs < chunks) cs *= 2;
    return launch_clusters(cache_dtype == VQ_E4M3 ? paged_compact_kernel<uint2> : paged_compact_kernel<uint4>, rows, cs,
                           MOVE_THREADS, 0, stream, p);
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
