// paged_keep_api.cpp - the extern "C" entry points that keep a part of a paged
// cache: argument validation, launches.  Host code only.
#include <cstdint>
#include <cstring>
#include <cuda_runtime_api.h>

#include "paged.h"
#include "paged_args.h"
#include "vq.h"

using namespace vq;

extern "C" {

vq_status vq_paged_select(const float *weights, int num_pages, int Hkv, int page_size, const int32_t *block_table,
                          int max_pages, const int32_t *lens, int B, int budget, int recent, int sinks, int32_t *keep,
                          int32_t *counts, vq_stream_t stream)
{
    const CacheArgs a = {nullptr, nullptr, nullptr, nullptr, VQ_F16, num_pages, Hkv, page_size};
    const vq_status st = check_cache_shape(a, kD);
    if (st != VQ_OK) return st;
    if (B < 0 || max_pages < 0 || budget < 0 || recent < 0 || sinks < 0 || (long long)recent + sinks > budget)
        return VQ_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > (1LL << 30) || budget > (1 << 30)) return VQ_ERR_UNSUPPORTED;
    if ((long long)B * Hkv > (1LL << 24)) return VQ_ERR_UNSUPPORTED;
    if (B == 0) return VQ_OK;
    if (!lens || !counts || (budget > 0 && !keep) || (max_pages > 0 && (!weights || !block_table))) return VQ_ERR_INVALID_ARG;
    if (!aligned(weights, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(keep, 4) || !aligned(counts, 4))
        return VQ_ERR_MISALIGNED;
    const Span outs[2] = {{keep, (size_t)B * Hkv * budget * 4}, {counts, (size_t)B * 4}};
    const Span ins[3] = {{weights, (size_t)a.rows() * 4}, {block_table, (size_t)B * max_pages * 4}, {lens, (size_t)B * 4}};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (overlap(o, i)) return VQ_ERR_ALIASING;
    if (overlap(outs[0], outs[1])) return VQ_ERR_ALIASING;
    PagedSelectParams p;
    std::memset(&p, 0, sizeof(p));
    p.weights = weights;
    p.table = block_table;
    p.lens = lens;
    p.keep = keep;
    p.counts = counts;
    p.num_pages = num_pages;
    p.Hkv = Hkv;
    p.page_shift = shift_of(page_size);
    p.B = B;
    p.max_pages = max_pages;
    p.budget = budget;
    p.recent = recent;
    p.sinks = sinks;
    return status_of(launch_paged_select(p, reinterpret_cast<cudaStream_t>(stream)));
}

vq_status vq_paged_compact(void *k_pages, void *v_pages, uint8_t *k_exp, uint8_t *v_exp, int cache_dtype, int num_pages,
                           int Hkv, int page_size, int D, const int32_t *block_table, int max_pages, const int32_t *keep,
                           long long keep_stride_b, long long keep_stride_h, int K, const int32_t *counts,
                           const int32_t *first, int B, float *weights, vq_stream_t stream)
{
    const CacheArgs a = {k_pages, v_pages, k_exp, v_exp, cache_dtype, num_pages, Hkv, page_size};
    vq_status st = check_cache_shape(a, D);
    if (st != VQ_OK) return st;
    if (B < 0 || K < 0 || max_pages < 0 || keep_stride_b < 0 || keep_stride_h < 0) return VQ_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > (1LL << 30) || K > (1 << 30)) return VQ_ERR_UNSUPPORTED;
    if ((long long)B * Hkv > (1LL << 24) || keep_stride_b >= (1LL << 38) || keep_stride_h >= (1LL << 38))
        return VQ_ERR_UNSUPPORTED;
    if (B == 0 || K == 0) return VQ_OK;
    if (!keep || !counts || !block_table || max_pages == 0 || num_pages == 0) return VQ_ERR_INVALID_ARG;
    if ((st = check_cache_ptrs(a, true, true)) != VQ_OK) return st;
    if (!aligned(keep, 4) || !aligned(counts, 4) || !aligned(first, 4) || !aligned(block_table, 4) || !aligned(weights, 4))
        return VQ_ERR_MISALIGNED;
    const Span outs[5] = {{k_pages, a.entry_bytes()}, {v_pages, a.entry_bytes()}, {a.exp_bytes() ? k_exp : nullptr, a.exp_bytes()},
                          {a.exp_bytes() ? v_exp : nullptr, a.exp_bytes()}, {weights, (size_t)a.rows() * 4}};
    const Span ins[4] = {{keep, ((size_t)(B - 1) * keep_stride_b + (size_t)(Hkv - 1) * keep_stride_h + K) * 4},
                         {counts, (size_t)B * 4}, {first, (size_t)B * 4}, {block_table, (size_t)B * max_pages * 4}};
    for (int i = 0; i < 5; ++i) {
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return VQ_ERR_ALIASING;
        for (int j = i + 1; j < 5; ++j)
            if (overlap(outs[i], outs[j])) return VQ_ERR_ALIASING;
    }
    PagedCompactParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = device_cache(a);
    p.table = block_table;
    p.keep = keep;
    p.keep_b = keep_stride_b;
    p.keep_h = keep_stride_h;
    p.counts = counts;
    p.first = first;
    p.weights = weights;
    p.B = B;
    p.max_pages = max_pages;
    p.K = K;
    return status_of(launch_paged_compact(p, cache_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
