// mla_softmax.cuh -- the arithmetic and warp-level pieces that the split kernel
// and the shared-prefix kernel have in common: powers of two, splitting values
// into e4m3 terms, reductions over a warp's keys, the softmax sets' barriers.
#pragma once
#include <cstdint>

#include "mla_sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

// 2^x by the hardware's approximation (relative error about 2^-22; results
// below the smallest normal fp32 flush to 0).
__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x * 2^k, exact whenever the result is a normal fp32 number.
__device__ __forceinline__ float mul_pow2(float x, int k)
{
    if (k > 127) {
        x *= __uint_as_float(254u << 23);
        k -= 127;
    } else if (k < -126) {
        x *= __uint_as_float(1u << 23);
        k += 126;
    }
    return x * __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Power-of-two shift that brings max |q| into [128, 256).
__device__ __forceinline__ int q_shift(float amax)
{
    if (!(amax > 0.f)) return 0;
    const uint32_t bits = __float_as_uint(amax);
    int e;  // amax = f * 2^e with f in [0.5, 1)
    if ((bits >> 23) != 0) e = (int)(bits >> 23) - 126;
    else frexpf(amax, &e);
    return 8 - e;
}

// Packed e4m3x2 -> two fp32 through the conversion unit (exact).
__device__ __forceinline__ float2 e4m3x2_to_f32x2_cvt(uint16_t v)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(v));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h2));
    return make_float2(lo, hi);
}

// Split two fp32 values into e4m3 hi bytes and e4m3 bytes of the residual
// times 2^kLoBits (pairs packed lo-byte first); returns the values the pairs
// represent, hi + lo * 2^-kLoBits (exact in fp32: the subtraction and the
// power-of-two scalings are exact).
template <int kLoBits>
__device__ __forceinline__ float2 split_pair(float a, float b, uint16_t& hi, uint16_t& lo)
{
    constexpr float up = (float)(1 << kLoBits);
    constexpr float back = 1.f / up;
    hi = f32x2_to_e4m3x2(a, b);
    const float2 h = e4m3x2_to_f32x2_cvt(hi);
    lo = f32x2_to_e4m3x2((a - h.x) * up, (b - h.y) * up);
    const float2 l = e4m3x2_to_f32x2_cvt(lo);
    return make_float2(fmaf(l.x, back, h.x), fmaf(l.y, back, h.y));
}

// Reduce N values held by every lane of a warp (max or sum); afterwards lane l
// holds the result for value index (l * N) / 32.
template <int N, bool MAX>
__device__ __forceinline__ float warp_transpose_reduce(float (&v)[N], int lane)
{
    int count = N;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        if (count > 1) {
            const int half = count >> 1;
            const bool upper = (lane & off) != 0;
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                if (k < half) {
                    const float send = upper ? v[k] : v[k + half];
                    const float keep = upper ? v[k + half] : v[k];
                    const float recv = __shfl_xor_sync(0xffffffffu, send, off);
                    v[k] = MAX ? fmaxf(keep, recv) : keep + recv;
                }
            }
            count = half;
        } else {
            const float recv = __shfl_xor_sync(0xffffffffu, v[0], off);
            v[0] = MAX ? fmaxf(v[0], recv) : v[0] + recv;
        }
    }
    return v[0];
}

// Barrier of the four warps of one softmax set (id 1 or 3, 128 threads).  Only
// used at points that all four warps of the set always reach.
__device__ __forceinline__ void softmax_bar(uint32_t id)
{
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

// The same barrier, returning the OR of `v` over the set's four warps.
__device__ __forceinline__ bool softmax_bar_or(uint32_t id, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %2, 0;\n\t"
        "bar.red.or.pred po, %1, 128, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

// Bounded wait whose outcome is the same on every lane of the warp (all lanes
// must call it), so no warp-collective instruction is reached divergently.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t sleep_ns = 0,
                                          long long limit = kWaitLimitCycles)
{
    const bool ok = mbar_wait_or_abort(bar, parity, abort, sleep_ns, limit);
    return __all_sync(0xffffffffu, ok);
}

}  // namespace
}  // namespace mla
