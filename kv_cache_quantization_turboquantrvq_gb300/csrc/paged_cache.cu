// paged_cache.cu - writing new tokens into a paged key/value cache and reading
// ranges of it back (sm_103a).
//
// Both move each byte once and compute almost nothing, so HBM bounds them: a
// row of 128 entries is taken by 16 lanes, 16 bytes of 16-bit entries each, and
// every access of a warp covers whole rows.
//
// The 8-bit cache holds x = code * 2^e with e4m3 codes and one exponent per
// token and head, the least with max|x| <= 448 * 2^e.  A power of two loses
// nothing against an exact scale (the codes are floating point, their relative
// step is the same over the whole range), x * 2^-e is exact, so a code is
// rounded once, and reading back is one exact product rounded to the output
// type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pc_err);

constexpr int THREADS = 256;

template <class T> struct Pair;
template <> struct Pair<__half> {
    using type = __half2;
    static __device__ __forceinline__ float2 f(__half2 v) { return __half22float2(v); }
    static __device__ __forceinline__ __half2 from(float2 v) { return __float22half2_rn(v); }
};
template <> struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ float2 f(__nv_bfloat162 v) { return __bfloat1622float2(v); }
    static __device__ __forceinline__ __nv_bfloat162 from(float2 v) { return __float22bfloat162_rn(v); }
};

// Exponent of a row from its largest magnitude (fp32 bits of a non-negative
// value): with max = m 2^f, 1 <= m < 2, the least e with m 2^f <= 1.75 * 2^(8 + e).
__device__ __forceinline__ int row_exponent(uint32_t bits)
{
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return bits == 0u ? 0 : min(max(e, PG_EMIN), PG_EMAX);
}

template <class T, bool E4M3>
__global__ void __launch_bounds__(THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams p)
{
    using T2 = typename Pair<T>::type;
    const int lane = threadIdx.x & 15;
    const long long row = (long long)blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4);  // (token, head)
    if (row >= (long long)p.T * p.c.Hkv) return;  // whole groups of 16 lanes leave together
    const int t = fdiv(p.divH, (int)row), h = (int)row - t * p.c.Hkv;
    const long long slot = __ldg(p.slots + t);
    if (slot < 0) return;  // a padding token
    const long long page = slot >> p.c.page_shift;
    if (page >= p.c.num_pages) {
        if (lane == 0) atomicOr(&g_pc_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        return;
    }
    const int off = (int)(slot - (page << p.c.page_shift));
    const long long dst = ((page * p.c.Hkv + h) << p.c.page_shift) + off;
    const unsigned group = 0xffffu << (threadIdx.x & 16);
    uint4 raw[2];
    raw[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_in) + t * p.kst + h * p.ksh) + lane);
    raw[1] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v_in) + t * p.vst + h * p.vsh) + lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        void *pages = const_cast<void *>(i ? p.c.v : p.c.k);
        if constexpr (!E4M3) {
            static_cast<uint4 *>(pages)[dst * 16 + lane] = raw[i];
        } else {
            const T2 *x = reinterpret_cast<const T2 *>(&raw[i]);
            float2 f[4];
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = Pair<T>::f(x[j]);
                m = fmaxf(m, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
            }
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, s));
            const int e = row_exponent(__float_as_uint(m));
            const float inv = pow2f(-e);
            uint2 code;
            uint16_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[j].x * inv, f[j].y * inv), __NV_SATFINITE, __NV_E4M3);
            code.x = (uint32_t)c[0] | ((uint32_t)c[1] << 16);
            code.y = (uint32_t)c[2] | ((uint32_t)c[3] << 16);
            static_cast<uint2 *>(pages)[dst * 16 + lane] = code;
            if (lane == 0) const_cast<uint8_t *>(i ? p.c.ve : p.c.ke)[dst] = (uint8_t)(e + 127);
        }
    }
}

template <class T, bool E4M3>
__device__ __forceinline__ uint4 read_row(const void *pages, const uint8_t *exps, long long src, int lane)
{
    if constexpr (!E4M3) {
        return __ldcs(static_cast<const uint4 *>(pages) + src * 16 + lane);
    } else {
        const uint2 code = __ldcs(static_cast<const uint2 *>(pages) + src * 16 + lane);
        const float s = pow2f((int)__ldg(exps + src) - 127);
        uint4 out;
        uint32_t *o = reinterpret_cast<uint32_t *>(&out);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t two = ((j < 2 ? code.x : code.y) >> (16 * (j & 1))) & 0xffffu;
            const uint32_t h2 = e4m3x2_to_f16x2(two);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            typename Pair<T>::type r = Pair<T>::from(make_float2(f.x * s, f.y * s));
            o[j] = *reinterpret_cast<uint32_t *>(&r);
        }
        return out;
    }
}

template <class T, bool E4M3>
__global__ void __launch_bounds__(THREADS) paged_gather_kernel(const __grid_constant__ PagedGatherParams p)
{
    const int lane = threadIdx.x & 15;
    const long long row = (long long)blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4);  // (b, h, i)
    if (row >= (long long)p.B * p.c.Hkv * p.S_out) return;
    const int bh = fdiv(p.divS, (int)row), i = (int)row - bh * p.S_out;
    const int b = fdiv(p.divH, bh), h = bh - b * p.c.Hkv;
    const long long t = (long long)(p.first ? __ldg(p.first + b) : 0) + i;
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (t >= 0 && t < __ldg(p.lens + b)) {
        const long long lp = t >> p.c.page_shift;
        const int page = lp < p.max_pages ? __ldg(p.table + (long long)b * p.max_pages + lp) : -1;
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) atomicOr(&g_pc_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        } else {
            const long long src =
                (((long long)page * p.c.Hkv + h) << p.c.page_shift) + (t & ((1 << p.c.page_shift) - 1));
            if (p.k_out) k = read_row<T, E4M3>(p.c.k, p.c.ke, src, lane);
            if (p.v_out) v = read_row<T, E4M3>(p.c.v, p.c.ve, src, lane);
        }
    }
    if (p.k_out) __stcs(static_cast<uint4 *>(p.k_out) + row * 16 + lane, k);
    if (p.v_out) __stcs(static_cast<uint4 *>(p.v_out) + row * 16 + lane, v);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams &p0, int in_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAppendParams p = p0;
    p.divH = make_fastdiv((uint32_t)p.c.Hkv);
    const long long rows = (long long)p.T * p.c.Hkv;
    const unsigned grid = (unsigned)((rows + THREADS / 16 - 1) / (THREADS / 16));
    const bool q = cache_dtype == VQ_E4M3;
    if (in_dtype == VQ_F16) {
        if (q) paged_append_kernel<__half, true><<<grid, THREADS, 0, stream>>>(p);
        else paged_append_kernel<__half, false><<<grid, THREADS, 0, stream>>>(p);
    } else {
        if (q) paged_append_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, stream>>>(p);
        else paged_append_kernel<__nv_bfloat16, false><<<grid, THREADS, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_paged_gather(const PagedGatherParams &p0, int cache_dtype, int out_dtype, cudaStream_t stream)
{
    PagedGatherParams p = p0;
    p.divH = make_fastdiv((uint32_t)p.c.Hkv);
    p.divS = make_fastdiv((uint32_t)p.S_out);
    const long long rows = (long long)p.B * p.c.Hkv * p.S_out;
    const unsigned grid = (unsigned)((rows + THREADS / 16 - 1) / (THREADS / 16));
    if (cache_dtype != VQ_E4M3) paged_gather_kernel<__half, false><<<grid, THREADS, 0, stream>>>(p);  // 16-bit copy
    else if (out_dtype == VQ_F16) paged_gather_kernel<__half, true><<<grid, THREADS, 0, stream>>>(p);
    else paged_gather_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t paged_cache_take_device_error(unsigned *bits, cudaStream_t stream)
{
    *bits = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_pc_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (*bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_pc_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace vq
