// paged_args.h - checks of the arguments that the paged-cache entry points
// share: views, caches, overlaps.  Host code only.
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

#include "paged.h"
#include "vq.h"

namespace vq {
namespace {

constexpr int kD = 128;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void *p;
    size_t n;
};

inline bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

inline bool is16(int t) { return t == VQ_F16 || t == VQ_BF16; }

// bytes from the first to the last element of a [T, H, 128] view of 16-bit elements
inline size_t view_bytes(long long T, int H, long long st, long long sh)
{
    return T <= 0 || H <= 0 ? 0 : (size_t)(((T - 1) * st + (H - 1) * sh + kD) * 2);
}

// A strided [T, H, 128] view that a kernel may read in 16-byte pieces.
inline vq_status check_view(const void *p, long long T, int H, long long st, long long sh)
{
    if (!p) return VQ_ERR_INVALID_ARG;
    if ((T > 1 && st < kD) || (H > 1 && sh < kD) || st < 0 || sh < 0) return VQ_ERR_INVALID_ARG;
    if (st >= (1LL << 38) || sh >= (1LL << 38)) return VQ_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || (T > 1 && st % 8 != 0) || (H > 1 && sh % 8 != 0)) return VQ_ERR_MISALIGNED;
    return VQ_OK;
}

inline int shift_of(int page_size)
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
inline vq_status check_cache_shape(const CacheArgs &a, int D)
{
    if (a.num_pages < 0 || a.Hkv <= 0 || D <= 0 || a.page_size <= 0) return VQ_ERR_INVALID_ARG;
    if (a.dtype != VQ_F16 && a.dtype != VQ_BF16 && a.dtype != VQ_E4M3) return VQ_ERR_INVALID_ARG;
    if (D != kD || shift_of(a.page_size) < 0) return VQ_ERR_UNSUPPORTED;
    if (a.rows() >= (1LL << 31)) return VQ_ERR_UNSUPPORTED;
    return VQ_OK;
}

inline vq_status check_cache_ptrs(const CacheArgs &a, bool k, bool v)
{
    const bool q = a.dtype == VQ_E4M3;
    if ((k && (!a.k || (q && !a.ke))) || (v && (!a.v || (q && !a.ve)))) return VQ_ERR_INVALID_ARG;
    if ((k && (!aligned(a.k, 16) || (q && !aligned(a.ke, 16)))) ||
        (v && (!aligned(a.v, 16) || (q && !aligned(a.ve, 16)))))
        return VQ_ERR_MISALIGNED;
    return VQ_OK;
}

inline PagedCache device_cache(const CacheArgs &a)
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

inline vq_status status_of(cudaError_t e) { return e == cudaSuccess ? VQ_OK : VQ_ERR_CUDA; }

inline size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace vq
