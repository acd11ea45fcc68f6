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

#include <type_traits>

#include "device_common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace vq {

namespace {

VQ_DEFINE_ERROR_WORD(g_pc_err);

constexpr int THREADS = 256;
// Rows a group of 16 lanes takes, their loads in flight together.  Measured at 1, 2
// and 4: 200000 tokens of 8 heads to codes 5643, 6071, 5734 GB/s, in 16 bits 6506,
// 6609, 6589; 4 x 32 x 32768 codes read back 6510, 6840, 6744.
constexpr int R = 2;

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

// R rows (token, head) a group of 16 lanes, all of their loads in flight at once.
template <class T, bool E4M3>
__global__ void __launch_bounds__(THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams p)
{
    using T2 = typename Pair<T>::type;
    const int lane = threadIdx.x & 15;
    const int rows = p.T * p.c.Hkv;  // below 2^31
    const long long r0 = ((long long)blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4)) * R;
    if (r0 >= rows) return;  // whole groups of 16 lanes leave together
    uint4 raw[R][2];
    long long slot[R];
    int head[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int row = (int)min(r0 + j, (long long)rows - 1);
        const int t = fdiv(p.divH, row), h = row - t * p.c.Hkv;
        head[j] = h;
        slot[j] = r0 + j < rows ? __ldg(p.slots + t) : -1;
        raw[j][0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_in) + t * p.kst + h * p.ksh) + lane);
        raw[j][1] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v_in) + t * p.vst + h * p.vsh) + lane);
    }
    const unsigned group = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (slot[j] < 0) continue;  // a padding token
        const long long page = slot[j] >> p.c.page_shift;
        if (page >= p.c.num_pages) {
            if (lane == 0) atomicOr(&g_pc_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
            continue;
        }
        const long long dst = ((page * p.c.Hkv + head[j]) << p.c.page_shift) + (slot[j] - (page << p.c.page_shift));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            void *pages = const_cast<void *>(i ? p.c.v : p.c.k);
            if constexpr (!E4M3) {
                static_cast<uint4 *>(pages)[dst * 16 + lane] = raw[j][i];
            } else {
                const T2 *x = reinterpret_cast<const T2 *>(&raw[j][i]);
                float2 f[4];
                float m = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f[q] = Pair<T>::f(x[q]);
                    m = fmaxf(m, fmaxf(fabsf(f[q].x), fabsf(f[q].y)));
                }
#pragma unroll
                for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, s));
                const int e = row_exponent(__float_as_uint(m));
                const float inv = pow2f(-e);
                uint16_t c[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    c[q] = __nv_cvt_float2_to_fp8x2(make_float2(f[q].x * inv, f[q].y * inv), __NV_SATFINITE, __NV_E4M3);
                static_cast<uint2 *>(pages)[dst * 16 + lane] =
                    make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16), (uint32_t)c[2] | ((uint32_t)c[3] << 16));
                if (lane == 0) const_cast<uint8_t *>(i ? p.c.ve : p.c.ke)[dst] = (uint8_t)(e + 127);
            }
        }
    }
}

// Eight entries of one 16-bit type as another: bf16 as fp16 (what the codecs take),
// rounded once to nearest, past 65504 to infinity.
__device__ __forceinline__ uint4 bf16x8_to_f16x8(uint4 v)
{
    auto two = [](uint32_t x) {
        const __half2 h = __float22half2_rn(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x)));
        return *reinterpret_cast<const uint32_t *>(&h);
    };
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

// R rows (tokens of one sequence and head) a group of 16 lanes, all of their
// loads in flight at once; S_out is padded to a multiple of R in the numbering.
// T: output type; KIND: what the pages hold.
enum { GATHER_SAME, GATHER_BF16, GATHER_E4M3 };
template <class T, int KIND>
__global__ void __launch_bounds__(THREADS) paged_gather_kernel(const __grid_constant__ PagedGatherParams p)
{
    constexpr bool E4M3 = KIND == GATHER_E4M3;
    using V = typename std::conditional<E4M3, uint2, uint4>::type;  // what 16 lanes of a row read
    const int lane = threadIdx.x & 15;
    const int blocks = (p.S_out + R - 1) / R;
    const long long at = (long long)blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4);
    if (at >= (long long)p.B * p.c.Hkv * blocks) return;
    const int bh = fdiv(p.divS, (int)at), i0 = ((int)at - bh * blocks) * R;
    const int b = fdiv(p.divH, bh), h = bh - b * p.c.Hkv;
    const long long t0 = (long long)(p.first ? __ldg(p.first + b) : 0) + i0;
    const int len = __ldg(p.lens + b);
    long long src[R];  // row of the pool, -1: none
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const long long t = t0 + j;
        src[j] = -1;
        if (i0 + j < p.S_out && t >= 0 && t < len) {
            const long long lp = t >> p.c.page_shift;
            const int page = lp < p.max_pages ? __ldg(p.table + (long long)b * p.max_pages + lp) : -1;
            if (page >= 0 && page < p.c.num_pages)
                src[j] = (((long long)page * p.c.Hkv + h) << p.c.page_shift) + (t & ((1 << p.c.page_shift) - 1));
            else if (lane == 0)
                atomicOr(&g_pc_err, (unsigned)VQ_DEVERR_BAD_OFFSET);
        }
    }
    V raw[R][2];
    uint8_t e[R][2];
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            raw[j][i] = V();
            e[j][i] = 127;
            if (src[j] >= 0 && (i ? p.v_out : p.k_out)) {
                raw[j][i] = __ldcs(static_cast<const V *>(i ? p.c.v : p.c.k) + src[j] * 16 + lane);
                if constexpr (E4M3) e[j][i] = __ldg((i ? p.c.ve : p.c.ke) + src[j]);
            }
        }
    }
    const long long dst = ((long long)bh * p.S_out + i0) * 16 + lane;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (i0 + j >= p.S_out) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            void *out = i ? p.v_out : p.k_out;
            if (!out) continue;
            uint4 x;
            if constexpr (E4M3) {
                const float s = pow2f((int)e[j][i] - 127);
                uint32_t h2[4];
                e4m3x4_to_f16x4(raw[j][i].x, h2[0], h2[1]);
                e4m3x4_to_f16x4(raw[j][i].y, h2[2], h2[3]);
                uint32_t *o = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2[q]));
                    const typename Pair<T>::type r = Pair<T>::from(make_float2(f.x * s, f.y * s));
                    o[q] = *reinterpret_cast<const uint32_t *>(&r);
                }
            } else if constexpr (KIND == GATHER_BF16) {
                x = bf16x8_to_f16x8(raw[j][i]);
            } else {
                x = raw[j][i];
            }
            __stcs(static_cast<uint4 *>(out) + dst + j * 16, x);
        }
    }
}

}  // namespace

namespace {

template <class T, bool E4M3> cudaError_t append(const PagedAppendParams &p, cudaStream_t stream)
{
    const long long rows = (long long)p.T * p.c.Hkv;
    const unsigned grid = (unsigned)((rows + R * (THREADS / 16) - 1) / (R * (THREADS / 16)));
    paged_append_kernel<T, E4M3><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <class T, int KIND> cudaError_t gather(PagedGatherParams &p, cudaStream_t stream)
{
    const int blocks = (p.S_out + R - 1) / R;
    p.divS = make_fastdiv((uint32_t)blocks);
    const long long groups = (long long)p.B * p.c.Hkv * blocks;
    paged_gather_kernel<T, KIND><<<(unsigned)((groups + THREADS / 16 - 1) / (THREADS / 16)), THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams &p0, int in_dtype, int cache_dtype, cudaStream_t stream)
{
    PagedAppendParams p = p0;
    p.divH = make_fastdiv((uint32_t)p.c.Hkv);
    if (cache_dtype != VQ_E4M3) return append<__half, false>(p, stream);  // 16-bit copy
    return in_dtype == VQ_F16 ? append<__half, true>(p, stream) : append<__nv_bfloat16, true>(p, stream);
}

cudaError_t launch_paged_gather(const PagedGatherParams &p0, int cache_dtype, int out_dtype, cudaStream_t stream)
{
    PagedGatherParams p = p0;
    p.divH = make_fastdiv((uint32_t)p.c.Hkv);
    if (cache_dtype == out_dtype) return gather<__half, GATHER_SAME>(p, stream);  // 16-bit copy
    if (cache_dtype == VQ_BF16) return gather<__half, GATHER_BF16>(p, stream);
    return out_dtype == VQ_F16 ? gather<__half, GATHER_E4M3>(p, stream) : gather<__nv_bfloat16, GATHER_E4M3>(p, stream);
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
