// paged_api.cpp - the extern "C" entry points of the paged-cache operators:
// argument validation, the workspace's layout, launches.  Host code only.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime_api.h>

#include "paged.h"
#include "paged_args.h"
#include "vq.h"

using namespace vq;

namespace {

constexpr int kMaxGroup = 16;  // query heads per kv head
constexpr size_t kPlanned = 256;  // at the workspace's end: the word that says the plan is made

// ------------------------------------------------- the attention's workspace

struct Layout {
    size_t start, cmb, ent, base, part, end;
};

// One class of entries from byte `at`; cap 0: the class is not used.
Layout layout(size_t at, int cap, int G, int rows)
{
    Layout l;
    l.start = at;
    l.cmb = l.start + up(cap ? sizeof(PgStart) * G : 0);
    l.ent = l.cmb + up(cap ? sizeof(int4) * G : 0);
    l.base = l.ent + up(sizeof(PgEntry) * (size_t)cap);
    l.part = l.base + up(sizeof(long long) * (size_t)cap);
    l.end = l.part + up(cap ? sizeof(float) * 2 * (size_t)G * rows * PG_PART : 0);
    return l;
}

struct AttendPlan {
    int small_rows, small_cap, small_tq, large_cap, large_tq, G;
    size_t bytes;
    Layout s, l;
    size_t planned, masks, depth;    // (trees)
    size_t wbase, lse, scores;       // (weights)
    int srows;
};

// keys (PG_WEIGH): tokens that the block table has room for.
vq_status attend_plan(int T, int B, int Hq, int Hkv, int max_q, PgMode mode, long long keys, AttendPlan &pl)
{
    if (T < 0 || B < 0 || Hq < 0 || Hkv <= 0 || max_q < 0 || Hq % Hkv != 0) return VQ_ERR_INVALID_ARG;
    const int gq = Hq / Hkv;
    if (gq > kMaxGroup) return VQ_ERR_UNSUPPORTED;
    if ((long long)T * Hq >= (1LL << 31) || B > (1 << 20)) return VQ_ERR_UNSUPPORTED;
    std::memset(&pl, 0, sizeof(pl));
    pl.G = sm_count() < PLAN_CTAS ? sm_count() : PLAN_CTAS;
    if (T == 0 || B == 0 || gq == 0) return VQ_OK;
    // Sequences with at most 16 query rows per kv head go to the small kernel,
    // longer chunks to the tensor-memory kernel.  A call whose bounds leave one
    // kind only (max_q short, or every sequence at max_q) launches one kernel.
    // The small kernel has a form for 8 rows, which is taken where it does: in
    // a call that launches the large kernel too, 9 to 16 rows go there.
    pl.small_tq = PG_SROWS / gq;
    pl.large_tq = 2 * (128 / gq);
    const bool large = (long long)max_q * gq > PG_SROWS;
    const bool small = !large || (long long)B * max_q > T;
    const bool narrow = large ? gq <= PG_SROWS / 2 : (long long)max_q * gq <= PG_SROWS / 2;
    pl.small_rows = !small ? 0 : narrow ? PG_SROWS / 2 : PG_SROWS;
    if (small) pl.small_cap = B;
    if (large) pl.large_cap = (T + pl.large_tq - 1) / pl.large_tq + B;
    pl.s = layout(0, pl.small_cap, pl.G, PG_SROWS);
    pl.l = layout(pl.s.end, pl.large_cap, pl.G, PG_LROWS);
    pl.planned = pl.l.end;
    pl.masks = pl.planned + (small && large ? kPlanned : 0);
    pl.depth = pl.masks + (mode == PG_TREE && large ? up((size_t)T * PG_TREE_WORDS * 4) : 0);
    pl.bytes = pl.depth + (mode == PG_TREE && large ? up((size_t)T * 4) : 0);
    if (mode == PG_WEIGH) {
        // scores of the small kernel's rows, or the parts of a chunk's sums
        pl.srows = !small ? 0 : pl.small_rows < (long long)max_q * gq ? pl.small_rows : max_q * gq;
        if (large && pl.srows < PG_PARTS) pl.srows = PG_PARTS;
        if ((double)B * Hkv * pl.srows * (double)keys >= 1e15) return VQ_ERR_UNSUPPORTED;
        pl.wbase = pl.bytes;
        pl.lse = pl.wbase + (large ? up((size_t)(B + 1) * 8) : 0);
        pl.scores = pl.lse + up((size_t)T * Hq * 4);
        pl.bytes = pl.scores + up((size_t)B * Hkv * pl.srows * (size_t)keys * 4);
    }
    return VQ_OK;
}

void place(PgPlan &d, unsigned char *ws, const Layout &l, int cap, int G, int tq)
{
    d.start = reinterpret_cast<PgStart *>(ws + l.start);
    d.cmb = reinterpret_cast<int4 *>(ws + l.cmb);
    d.ent = reinterpret_cast<PgEntry *>(ws + l.ent);
    d.base = reinterpret_cast<long long *>(ws + l.base);
    d.part = reinterpret_cast<float *>(ws + l.part);
    d.cap = cap;
    d.G = G;
    d.tq = tq;
}

// What a call's new tokens are besides the next ones in order.
struct AttendExtra {
    PgMode mode;
    const int32_t *parents;  // PG_TREE
    float *weights;          // PG_WEIGH
    int observe;
    float decay;
};

vq_status attend(const AttendExtra &x, const CacheArgs &a, int D, const void *q, long long q_stride_t, long long q_stride_h,
                 int q_dtype, const int32_t *block_table, int max_pages, const int32_t *cu_q, const int32_t *lens, int T,
                 int B, int Hq, int max_q, int window, int sinks, float scale, void *out, void *workspace,
                 size_t workspace_bytes, vq_stream_t stream)
{
    const int Hkv = a.Hkv, num_pages = a.num_pages, page_size = a.page_size, cache_dtype = a.dtype;
    vq_status st = check_cache_shape(a, D);
    if (st != VQ_OK) return st;
    AttendPlan pl;
    if ((st = attend_plan(T, B, Hq, Hkv, max_q, x.mode, (long long)(max_pages > 0 ? max_pages : 0) * page_size, pl)) != VQ_OK) return st;
    const float qscale = (float)((double)scale * 1.4426950408889634);  // the kernels' exponents are of base 2
    if (!is16(q_dtype) || max_pages < 0 || window < 0 || sinks < 0 || !std::isfinite(qscale)) return VQ_ERR_INVALID_ARG;
    if (cache_dtype != VQ_E4M3 && cache_dtype != q_dtype) return VQ_ERR_INVALID_ARG;
    // (positions and a window behind them stay within 32 bits)
    if ((long long)max_pages * page_size > (1LL << 30) || T > (1 << 30)) return VQ_ERR_UNSUPPORTED;
    if (x.mode == PG_TREE && max_q > PG_TREE_MAX) return VQ_ERR_UNSUPPORTED;
    if (x.mode == PG_WEIGH && (x.observe < 0 || !(x.decay >= 0.0f && x.decay <= 1.0f))) return VQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || Hq == 0) return VQ_OK;
    if (max_q == 0) return VQ_ERR_INVALID_ARG;
    if ((st = check_view(q, T, Hq, q_stride_t, q_stride_h)) != VQ_OK) return st;
    // an empty pool or table: no key is visible, but the maps need an address
    if (num_pages == 0 || max_pages == 0) return VQ_ERR_INVALID_ARG;
    if ((st = check_cache_ptrs(a, true, true)) != VQ_OK) return st;
    if (!block_table || !cu_q || !lens || !out || !workspace) return VQ_ERR_INVALID_ARG;
    if ((x.mode == PG_TREE && !x.parents) || (x.mode == PG_WEIGH && !x.weights)) return VQ_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(lens, 4) || !aligned(out, 16) || !aligned(workspace, 256) ||
        !aligned(x.parents, 4) || !aligned(x.weights, 16))
        return VQ_ERR_MISALIGNED;
    if (workspace_bytes < pl.bytes) return VQ_ERR_INVALID_ARG;
    const Span outs[3] = {{out, (size_t)T * Hq * kD * 2}, {workspace, pl.bytes}, {x.weights, (size_t)a.rows() * 4}};
    const Span ins[9] = {{q, view_bytes(T, Hq, q_stride_t, q_stride_h)}, {a.k, a.entry_bytes()},
                         {a.v, a.entry_bytes()}, {a.exp_bytes() ? a.ke : nullptr, a.exp_bytes()},
                         {a.exp_bytes() ? a.ve : nullptr, a.exp_bytes()},
                         {block_table, (size_t)B * max_pages * 4}, {cu_q, (size_t)(B + 1) * 4}, {lens, (size_t)B * 4},
                         {x.parents, (size_t)T * 4}};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (overlap(o, i)) return VQ_ERR_ALIASING;
    if (overlap(outs[0], outs[1]) || overlap(outs[0], outs[2]) || overlap(outs[1], outs[2])) return VQ_ERR_ALIASING;

    PagedAttendParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = device_cache(a);
    p.q = q;
    p.qst = q_stride_t;
    p.qsh = q_stride_h;
    p.table = block_table;
    p.cu = cu_q;
    p.lens = lens;
    p.out = out;
    p.T = T;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.GQ = Hq / Hkv;
    p.max_pages = max_pages;
    p.max_q = max_q;
    p.window = window <= (long long)max_pages * page_size ? window : 0;  // (longer than any sequence: none)
    p.sinks = sinks;
    p.small_rows = pl.small_rows;
    p.qscale = qscale;
    // (scale 0: any factor that makes every finite score vanish, so that the
    // mask's -inf times it stays -inf)
    if (p.qscale == 0.0f) p.qscale = 1e-30f;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    place(p.small, ws, pl.s, pl.small_cap, pl.G, pl.small_tq);
    place(p.large, ws, pl.l, pl.large_cap, pl.G, pl.large_tq);
    if (pl.small_cap && pl.large_cap) {
        static std::atomic<unsigned long long> calls{0};
        p.planned = reinterpret_cast<unsigned long long *>(ws + pl.planned);
        p.call = ++calls;
    }
    if (x.mode == PG_TREE) {
        p.parents = x.parents;
        p.masks = reinterpret_cast<uint32_t *>(ws + pl.masks);
        p.depth = reinterpret_cast<int32_t *>(ws + pl.depth);
    }
    if (x.mode == PG_WEIGH) {
        p.wbase = pl.large_cap ? reinterpret_cast<long long *>(ws + pl.wbase) : nullptr;
        p.lse = reinterpret_cast<float *>(ws + pl.lse);
        p.scores = reinterpret_cast<float *>(ws + pl.scores);
        p.srows = pl.srows;
        p.keys = max_pages * page_size;
        p.weights = x.weights;
        p.decay = x.decay;
        p.observe = x.observe;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // (a call of small sequences alone: its kernel makes the plan)
    cudaError_t e = pl.large_cap ? launch_paged_plan(p, s) : cudaSuccess;
    if (e == cudaSuccess && pl.large_cap) e = launch_paged_large(p, q_dtype, cache_dtype, s);
    if (e == cudaSuccess && pl.small_cap) e = launch_paged_small(p, q_dtype, cache_dtype, s);
    if (e == cudaSuccess) e = launch_paged_combine(p, q_dtype, s);
    if (e == cudaSuccess && x.mode == PG_WEIGH && pl.large_cap) e = launch_paged_weigh(p, q_dtype, cache_dtype, s);
    if (e == cudaSuccess && x.mode == PG_WEIGH) e = launch_paged_weigh_update(p, s);
    return status_of(e);
}

}  // namespace

extern "C" {

vq_status vq_paged_append(const void *k_in, long long k_stride_t, long long k_stride_h, const void *v_in,
                          long long v_stride_t, long long v_stride_h, int in_dtype, int T, const int64_t *slots,
                          void *k_pages, void *v_pages, uint8_t *k_exp, uint8_t *v_exp, int cache_dtype,
                          int num_pages, int Hkv, int page_size, int D, vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    vq_status st = check_cache_shape(a, D);
    if (st != VQ_OK) return st;
    if (T < 0 || !is16(in_dtype)) return VQ_ERR_INVALID_ARG;
    if (cache_dtype != VQ_E4M3 && cache_dtype != in_dtype) return VQ_ERR_INVALID_ARG;
    if ((long long)T * Hkv >= (1LL << 31)) return VQ_ERR_UNSUPPORTED;
    if (T == 0) return VQ_OK;
    if ((st = check_view(k_in, T, Hkv, k_stride_t, k_stride_h)) != VQ_OK) return st;
    if ((st = check_view(v_in, T, Hkv, v_stride_t, v_stride_h)) != VQ_OK) return st;
    if ((st = check_cache_ptrs(a, true, true)) != VQ_OK) return st;
    if (!slots) return VQ_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return VQ_ERR_MISALIGNED;
    const Span outs[4] = {{k_pages, a.entry_bytes()}, {v_pages, a.entry_bytes()}, {a.exp_bytes() ? k_exp : nullptr, a.exp_bytes()},
                          {a.exp_bytes() ? v_exp : nullptr, a.exp_bytes()}};
    const Span ins[3] = {{k_in, view_bytes(T, Hkv, k_stride_t, k_stride_h)},
                         {v_in, view_bytes(T, Hkv, v_stride_t, v_stride_h)}, {slots, (size_t)T * 8}};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return VQ_ERR_ALIASING;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return VQ_ERR_ALIASING;
    }
    PagedAppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = device_cache(a);
    p.k_in = k_in;
    p.v_in = v_in;
    p.kst = k_stride_t;
    p.ksh = k_stride_h;
    p.vst = v_stride_t;
    p.vsh = v_stride_h;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.T = T;
    return status_of(launch_paged_append(p, in_dtype, cache_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

vq_status vq_paged_gather(const void *k_pages, const void *v_pages, const uint8_t *k_exp, const uint8_t *v_exp,
                          int cache_dtype, int num_pages, int Hkv, int page_size, int D, const int32_t *block_table,
                          int max_pages, const int32_t *lens, const int32_t *first, int B, int S_out, int out_dtype,
                          void *k_out, void *v_out, vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    vq_status st = check_cache_shape(a, D);
    if (st != VQ_OK) return st;
    if (B < 0 || S_out < 0 || max_pages < 0 || !is16(out_dtype)) return VQ_ERR_INVALID_ARG;
    if (cache_dtype == VQ_F16 && out_dtype != VQ_F16) return VQ_ERR_INVALID_ARG;
    if (!k_out && !v_out) return VQ_ERR_INVALID_ARG;
    if ((long long)B * Hkv * S_out >= (1LL << 31)) return VQ_ERR_UNSUPPORTED;
    if ((long long)B * S_out == 0) return VQ_OK;
    if (!lens || (max_pages > 0 && !block_table)) return VQ_ERR_INVALID_ARG;
    if ((st = check_cache_ptrs(a, k_out != nullptr && num_pages > 0, v_out != nullptr && num_pages > 0)) != VQ_OK) return st;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(lens, 4) || !aligned(first, 4) || !aligned(block_table, 4))
        return VQ_ERR_MISALIGNED;
    const size_t ob = (size_t)B * Hkv * S_out * kD * 2;
    const Span outs[2] = {{k_out, ob}, {v_out, ob}};
    const Span ins[7] = {{k_pages, a.entry_bytes()}, {v_pages, a.entry_bytes()},
                         {a.exp_bytes() ? k_exp : nullptr, a.exp_bytes()}, {a.exp_bytes() ? v_exp : nullptr, a.exp_bytes()},
                         {block_table, (size_t)B * max_pages * 4}, {lens, (size_t)B * 4}, {first, (size_t)B * 4}};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (overlap(o, i)) return VQ_ERR_ALIASING;
    if (overlap(outs[0], outs[1])) return VQ_ERR_ALIASING;
    PagedGatherParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = device_cache(a);
    p.table = block_table;
    p.lens = lens;
    p.first = first;
    p.k_out = k_out;
    p.v_out = v_out;
    p.B = B;
    p.max_pages = max_pages;
    p.S_out = S_out;
    return status_of(launch_paged_gather(p, cache_dtype, out_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

vq_status vq_paged_attend_workspace(int T, int B, int Hq, int Hkv, int max_q, size_t *bytes)
{
    if (!bytes) return VQ_ERR_INVALID_ARG;
    AttendPlan pl;
    const vq_status st = attend_plan(T, B, Hq, Hkv, max_q, PG_CHAIN, 0, pl);
    if (st != VQ_OK) return st;
    *bytes = pl.bytes;
    return VQ_OK;
}

vq_status vq_paged_attend(const void *q, long long q_stride_t, long long q_stride_h, int q_dtype,
                          const void *k_pages, const void *v_pages, const uint8_t *k_exp, const uint8_t *v_exp,
                          int cache_dtype, int num_pages, int Hkv, int page_size, int D, const int32_t *block_table,
                          int max_pages, const int32_t *cu_q, const int32_t *lens, int T, int B, int Hq, int max_q,
                          int window, int sinks, float scale, void *out, void *workspace, size_t workspace_bytes,
                          vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    return attend({PG_CHAIN, nullptr, nullptr, 0, 0.0f}, a, D, q, q_stride_t, q_stride_h, q_dtype, block_table, max_pages, cu_q, lens, T, B, Hq,
                  max_q, window, sinks, scale, out, workspace, workspace_bytes, stream);
}

vq_status vq_paged_attend_tree_workspace(int T, int B, int Hq, int Hkv, int max_q, size_t *bytes)
{
    if (!bytes) return VQ_ERR_INVALID_ARG;
    AttendPlan pl;
    const vq_status st = attend_plan(T, B, Hq, Hkv, max_q, PG_TREE, 0, pl);
    if (st != VQ_OK) return st;
    if (max_q > PG_TREE_MAX) return VQ_ERR_UNSUPPORTED;
    *bytes = pl.bytes;
    return VQ_OK;
}

vq_status vq_paged_attend_tree(const void *q, long long q_stride_t, long long q_stride_h, int q_dtype,
                               const void *k_pages, const void *v_pages, const uint8_t *k_exp, const uint8_t *v_exp,
                               int cache_dtype, int num_pages, int Hkv, int page_size, int D, const int32_t *block_table,
                               int max_pages, const int32_t *cu_q, const int32_t *lens, const int32_t *parents, int T, int B,
                               int Hq, int max_q, int window, int sinks, float scale, void *out, void *workspace,
                               size_t workspace_bytes, vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    return attend({PG_TREE, parents, nullptr, 0, 0.0f}, a, D, q, q_stride_t, q_stride_h, q_dtype, block_table, max_pages, cu_q, lens, T, B, Hq,
                  max_q, window, sinks, scale, out, workspace, workspace_bytes, stream);
}

vq_status vq_paged_attend_weigh_workspace(int T, int B, int Hq, int Hkv, int max_q, int max_pages, int page_size, size_t *bytes)
{
    if (!bytes || max_pages < 0) return VQ_ERR_INVALID_ARG;
    if (shift_of(page_size) < 0 || (long long)max_pages * page_size > (1LL << 30)) return VQ_ERR_UNSUPPORTED;
    AttendPlan pl;
    const vq_status st = attend_plan(T, B, Hq, Hkv, max_q, PG_WEIGH, (long long)max_pages * page_size, pl);
    if (st != VQ_OK) return st;
    *bytes = pl.bytes;
    return VQ_OK;
}

vq_status vq_paged_attend_weigh(const void *q, long long q_stride_t, long long q_stride_h, int q_dtype,
                                const void *k_pages, const void *v_pages, const uint8_t *k_exp, const uint8_t *v_exp,
                                int cache_dtype, int num_pages, int Hkv, int page_size, int D, const int32_t *block_table,
                                int max_pages, const int32_t *cu_q, const int32_t *lens, int T, int B, int Hq, int max_q,
                                int window, int sinks, float scale, float *weights, int observe, float decay, void *out,
                                void *workspace, size_t workspace_bytes, vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    return attend({PG_WEIGH, nullptr, weights, observe, decay}, a, D, q, q_stride_t, q_stride_h, q_dtype, block_table, max_pages,
                  cu_q, lens, T, B, Hq, max_q, window, sinks, scale, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
