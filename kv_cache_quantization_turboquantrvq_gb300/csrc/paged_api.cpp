// paged_api.cpp - the extern "C" entry points of the paged-cache operators:
// argument validation, the workspace's layout, launches.  Host code only.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime_api.h>

#include "paged.h"
#include "vq.h"

using namespace vq;

namespace {

constexpr int kD = 128;
constexpr int kMaxGroup = 16;  // query heads per kv head
constexpr size_t kPlanned = 256;  // at the workspace's end: the word that says the plan is made

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void *p;
    size_t n;
};

bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

bool is16(int t) { return t == VQ_F16 || t == VQ_BF16; }

// bytes from the first to the last element of a [T, H, 128] view of 16-bit elements
size_t view_bytes(long long T, int H, long long st, long long sh)
{
    return T <= 0 || H <= 0 ? 0 : (size_t)(((T - 1) * st + (H - 1) * sh + kD) * 2);
}

// A strided [T, H, 128] view that a kernel may read in 16-byte pieces.
vq_status check_view(const void *p, long long T, int H, long long st, long long sh)
{
    if (!p) return VQ_ERR_INVALID_ARG;
    if ((T > 1 && st < kD) || (H > 1 && sh < kD) || st < 0 || sh < 0) return VQ_ERR_INVALID_ARG;
    if (st >= (1LL << 38) || sh >= (1LL << 38)) return VQ_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || (T > 1 && st % 8 != 0) || (H > 1 && sh % 8 != 0)) return VQ_ERR_MISALIGNED;
    return VQ_OK;
}

int shift_of(int page_size)
{
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

struct CacheArgs {
    const void *k, *v;
    const uint8_t *ke, *ve;
    int dtype, num_pages, Hkv, page_size;
    long long rows() const { return (long long)num_pages * Hkv * page_size; }
    size_t entry_bytes() const { return (size_t)rows() * kD * (dtype == VQ_E4M3 ? 1 : 2); }
    size_t exp_bytes() const { return dtype == VQ_E4M3 ? (size_t)rows() : 0; }
};

// shape and type of a cache; `k` / `v`: which parts are needed
vq_status check_cache_shape(const CacheArgs &a, int D)
{
    if (a.num_pages < 0 || a.Hkv <= 0 || D <= 0 || a.page_size <= 0) return VQ_ERR_INVALID_ARG;
    if (a.dtype != VQ_F16 && a.dtype != VQ_BF16 && a.dtype != VQ_E4M3) return VQ_ERR_INVALID_ARG;
    if (D != kD || shift_of(a.page_size) < 0) return VQ_ERR_UNSUPPORTED;
    if (a.rows() >= (1LL << 31)) return VQ_ERR_UNSUPPORTED;
    return VQ_OK;
}

vq_status check_cache_ptrs(const CacheArgs &a, bool k, bool v)
{
    const bool q = a.dtype == VQ_E4M3;
    if ((k && (!a.k || (q && !a.ke))) || (v && (!a.v || (q && !a.ve)))) return VQ_ERR_INVALID_ARG;
    if ((k && (!aligned(a.k, 16) || (q && !aligned(a.ke, 16)))) ||
        (v && (!aligned(a.v, 16) || (q && !aligned(a.ve, 16)))))
        return VQ_ERR_MISALIGNED;
    return VQ_OK;
}

PagedCache device_cache(const CacheArgs &a)
{
    PagedCache c;
    c.k = a.k;
    c.v = a.v;
    c.ke = a.dtype == VQ_E4M3 ? a.ke : nullptr;
    c.ve = a.dtype == VQ_E4M3 ? a.ve : nullptr;
    c.num_pages = a.num_pages;
    c.Hkv = a.Hkv;
    c.page_shift = shift_of(a.page_size);
    return c;
}

vq_status status_of(cudaError_t e) { return e == cudaSuccess ? VQ_OK : VQ_ERR_CUDA; }

// ------------------------------------------------- the attention's workspace

size_t up(size_t n) { return (n + 255) / 256 * 256; }

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
};

vq_status attend_plan(int T, int B, int Hq, int Hkv, int max_q, AttendPlan &pl)
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
    pl.bytes = pl.l.end + (small && large ? kPlanned : 0);
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
    const vq_status st = attend_plan(T, B, Hq, Hkv, max_q, pl);
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
    vq_status st = check_cache_shape(a, D);
    if (st != VQ_OK) return st;
    AttendPlan pl;
    if ((st = attend_plan(T, B, Hq, Hkv, max_q, pl)) != VQ_OK) return st;
    const float qscale = (float)((double)scale * 1.4426950408889634);  // the kernels' exponents are of base 2
    if (!is16(q_dtype) || max_pages < 0 || window < 0 || sinks < 0 || !std::isfinite(qscale)) return VQ_ERR_INVALID_ARG;
    if (cache_dtype != VQ_E4M3 && cache_dtype != q_dtype) return VQ_ERR_INVALID_ARG;
    // (positions and a window behind them stay within 32 bits)
    if ((long long)max_pages * page_size > (1LL << 30) || T > (1 << 30)) return VQ_ERR_UNSUPPORTED;
    if (T == 0 || B == 0 || Hq == 0) return VQ_OK;
    if (max_q == 0) return VQ_ERR_INVALID_ARG;
    if ((st = check_view(q, T, Hq, q_stride_t, q_stride_h)) != VQ_OK) return st;
    // an empty pool or table: no key is visible, but the maps need an address
    if (num_pages == 0 || max_pages == 0) return VQ_ERR_INVALID_ARG;
    if ((st = check_cache_ptrs(a, true, true)) != VQ_OK) return st;
    if (!block_table || !cu_q || !lens || !out || !workspace) return VQ_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(lens, 4) || !aligned(out, 16) || !aligned(workspace, 256))
        return VQ_ERR_MISALIGNED;
    if (workspace_bytes < pl.bytes) return VQ_ERR_INVALID_ARG;
    const Span outs[2] = {{out, (size_t)T * Hq * kD * 2}, {workspace, pl.bytes}};
    const Span ins[8] = {{q, view_bytes(T, Hq, q_stride_t, q_stride_h)}, {k_pages, a.entry_bytes()},
                         {v_pages, a.entry_bytes()}, {a.exp_bytes() ? k_exp : nullptr, a.exp_bytes()},
                         {a.exp_bytes() ? v_exp : nullptr, a.exp_bytes()},
                         {block_table, (size_t)B * max_pages * 4}, {cu_q, (size_t)(B + 1) * 4}, {lens, (size_t)B * 4}};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (overlap(o, i)) return VQ_ERR_ALIASING;
    if (overlap(outs[0], outs[1])) return VQ_ERR_ALIASING;

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
        p.planned = reinterpret_cast<unsigned long long *>(ws + pl.l.end);
        p.call = ++calls;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // (a call of small sequences alone: its kernel makes the plan)
    cudaError_t e = pl.large_cap ? launch_paged_plan(p, s) : cudaSuccess;
    if (e == cudaSuccess && pl.large_cap) e = launch_paged_large(p, q_dtype, cache_dtype, s);
    if (e == cudaSuccess && pl.small_cap) e = launch_paged_small(p, q_dtype, cache_dtype, s);
    if (e == cudaSuccess) e = launch_paged_combine(p, q_dtype, s);
    return status_of(e);
}

}  // extern "C"
