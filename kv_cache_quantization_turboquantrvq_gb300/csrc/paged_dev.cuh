// paged_dev.cuh - device helpers of the paged-cache operators: e4m3 codes,
// powers of two, the walk over a launch's units of work.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "paged.h"

namespace vq {
namespace {

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four codes as two fp16 pairs; exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

constexpr uint32_t PG_EXP0 = 0x7f7f7f7fu;  // exponent 0 of four rows, as stored

// Exponents (a byte each) of four consecutive value rows of codes, those of zero
// rows replaced by the least one.  A zero row is stored with exponent 0, as if
// it were larger than the rows around it; it adds nothing to an output, so the
// softmax must not make room for it.  The codes are read only of rows with
// exponent 0, which are zero or reach beyond 224.
__device__ __forceinline__ uint32_t pg_value_exps(uint32_t four, const void *rows)
{
    const uint4 *row = static_cast<const uint4 *>(rows);
    const uint32_t ask = __vcmpeq4(four, PG_EXP0);
    auto some = [&](int i) {  // of 16 codes, without the signs
        const uint4 u = __ldg(row + i);
        return ((u.x | u.y | u.z | u.w) & 0x7f7f7f7fu) != 0u;
    };
    // most rows show within their first 16 codes that they are not zero
    uint32_t zero = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((ask >> (8 * i)) & 1u) zero |= some(8 * i) ? 0u : 0xffu << (8 * i);
    if (zero == 0u) return four;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        if (((zero >> (8 * i)) & 1u) == 0u) continue;
        bool any = false;
#pragma unroll
        for (int c = 1; c < 8; ++c) any |= some(8 * i + c);
        if (any) zero &= ~(0xffu << (8 * i));
    }
    return (four & ~zero) | (zero & (0x01010101u * (uint32_t)(PG_EMIN + 127)));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane of the (whole, converged) warp, the same each time.  Copies and
// products issued under it keep their operands in uniform registers.
__device__ __forceinline__ bool elect_lane()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
    return e != 0;
}

// Programmatic launch order: pg_wait() until the kernel before in the stream is
// complete and its writes are seen, pg_go() lets the next one start early (it
// takes the SMs as they become free).
__device__ __forceinline__ void pg_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pg_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A word written after, and read before, other memory by kernels that overlap.
__device__ __forceinline__ void pg_release(unsigned long long *at, unsigned long long v)
{
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long pg_acquire(const unsigned long long *at)
{
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
    return v;
}

// Barrier of the first THREADS threads of the CTA.
template <int THREADS> __device__ __forceinline__ void bar_compute()
{
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// What of an entry's keys its rows see together: [lo, hi) and the first `sink` keys.
struct PgView {
    int hi, lo, sink;
    __device__ __forceinline__ void set(const PgEntry &e, int window, int sinks)
    {
        hi = e.hi;
        lo = window > 0 ? max(0, e.p0 - window + 1) : 0;
        sink = window > 0 ? min(sinks, hi) : 0;
    }
    // some / every key of [k0, k1) is seen by some row
    __device__ __forceinline__ bool any(int k0, int k1) const { return k0 < hi && (k1 > lo || k0 < sink); }
    __device__ __forceinline__ bool one(int k) const { return k < hi && (k >= lo || k < sink); }
};

__device__ __forceinline__ PgEntry pg_entry(const PgEntry *e)
{
    const int4 a = *reinterpret_cast<const int4 *>(e), b = *(reinterpret_cast<const int4 *>(e) + 1);
    PgEntry r;
    r.b = a.x; r.tok0 = a.y; r.nt = a.z; r.p0 = a.w;
    r.hi = b.x; r.nsink = b.y; r.tl = b.z; r.ntiles = b.w;
    return r;
}

// first key of tile t of an entry
__device__ __forceinline__ int pg_tile_key(const PgEntry &e, int t)
{
    return (t < e.nsink ? t : e.tl + (t - e.nsink)) * PG_TILE;
}

// One CTA's share as runs of tiles of one item each.
struct PgRun {
    PgEntry e;
    int ei, h, t0, tn, left;
    bool first;  // the CTA's first run
    __device__ __forceinline__ void start(const PgStart &s)
    {
        const int4 at = *reinterpret_cast<const int4 *>(&s);
        e = pg_entry(&s.e);
        ei = at.x;
        h = at.y;
        t0 = at.z;
        left = at.w;  // 0: nothing to do
        tn = min(e.ntiles, t0 + left);
        first = true;
    }
    template <class F> __device__ __forceinline__ bool next(int Hkv, F &&step)  // step: to the next entry
    {
        left -= tn - t0;
        if (left <= 0) return false;
        if (++h == Hkv) {
            h = 0;
            step(*this);
        }
        t0 = 0;
        tn = min(e.ntiles, left);
        first = false;
        return true;
    }
    __device__ __forceinline__ bool next(const PgPlan &pl, int Hkv)
    {
        return next(Hkv, [&](PgRun &r) { r.e = pg_entry(pl.ent + ++r.ei); });
    }
};

// Position in a ring of N barriers: slot and the parity of its current pass.
template <int N> struct PgRing {
    int s = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void step()
    {
        if (++s == N) {
            s = 0;
            par ^= 1u;
        }
    }
};

}  // namespace
}  // namespace vq
