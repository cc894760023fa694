// tcg_lm_math.cuh -- device helpers shared by the kernels of the language-model products:
// packed FP32 arithmetic, activations and their slopes, 16-bit conversions, group ranges.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tcg_lm.h"
#include "tcg_ptx.cuh"

namespace tcg {

// ------------------------------------------------------------------------- activations
// Two FP32 values in a register pair: one instruction adds, multiplies or multiply-adds both
// (each rounded to nearest as the scalar forms).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split2(F2 p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
template <typename F>
__device__ __forceinline__ F2 each(F2 p, F f)
{
    float a, b;
    split2(p, a, b);
    return f2(f(a), f(b));
}

// 2^x and 1 / x on the special-function unit: relative error about 2^-22, results below
// 2^-126 flushed to zero.  That is under the rounding of every output type but FP32, where
// it is of the rounding's own size.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 exp2_2(F2 x) { return each(x, exp2_fast); }
__device__ __forceinline__ F2 rcp_2(F2 x) { return each(x, rcp_fast); }

constexpr float kLog2e = 1.4426950408889634f;

// erfc(|x| / sqrt 2) / 2 and gauss = exp(-x^2 / 2), ax = min(|x|, 20), past which both are
// zero.  The quotient of the two is smooth in t = 1 / (1 + 0.361 |x|): t times a polynomial of
// degree 6, fitted over |x| <= 13.5 for the least maximum of its error relative to the quotient
// (7.3e-7).  So the tail is right to its own size where FP32 holds it: within 1.3e-6 of itself,
// and x^2 7.5e-8 for the rounded argument of gauss.  (A fit of the absolute error has two terms
// fewer, but is off by 5e-5 of itself at -3 and by 1% at -8.)
__device__ __forceinline__ F2 half_erfc(F2 ax, F2 &gauss)
{
    const F2 t = rcp_2(fma2(f2(0.361f), ax, f2(1.0f)));
    gauss = exp2_2(ax * ax * f2(-0.5f * kLog2e));
    F2 q = fma2(t, f2(0.0477842689f), f2(-0.180867106f));
    q = fma2(t, q, f2(0.180101722f));
    q = fma2(t, q, f2(0.026798008f));
    q = fma2(t, q, f2(0.139898449f));
    q = fma2(t, q, f2(0.142172173f));
    q = fma2(t, q, f2(0.144112632f));
    return q * t * gauss;
}

template <int ACT>
__device__ __forceinline__ F2 act_fn(F2 x)
{
    if constexpr (ACT == kActRelu) {
        return each(x, [](float v) { return v < 0.0f ? 0.0f : v; });
    } else if constexpr (ACT == kActGelu) {
        // x Phi(x) = max(x, 0) - |x| erfc(|x| / sqrt 2) / 2; 0 x keeps NaN (and -inf, whose
        // product with zero has no value either)
        F2 g;
        const F2 ax = each(x, [](float v) { return fminf(fabsf(v), 20.0f); });
        const F2 h = half_erfc(ax, g);
        const F2 pos = each(x, [](float v) { return v > 0.0f ? v : 0.0f * v; });
        return fma2(ax * f2(-1.0f), h, pos);
    } else if constexpr (ACT == kActGeluTanh) {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3)
        const F2 c = f2(-1.5957691216057308f * kLog2e);
        const F2 e = exp2_2(x * fma2(c * f2(0.044715f) * x, x, c));
        return x * rcp_2(e + f2(1.0f));
    } else if constexpr (ACT == kActSilu) {
        return x * rcp_2(exp2_2(x * f2(-kLog2e)) + f2(1.0f));
    } else {
        return x;
    }
}

template <int ACT>
__device__ __forceinline__ F2 act_slope(F2 x)
{
    if constexpr (ACT == kActRelu) {
        return each(x, [](float v) { return v > 0.0f ? 1.0f : (v <= 0.0f ? 0.0f : v); });
    } else if constexpr (ACT == kActGelu) {
        F2 g;
        const F2 ax = each(x, [](float v) { return fminf(fabsf(v), 20.0f); });
        float h0, h1, x0, x1;
        split2(half_erfc(ax, g), h0, h1);
        split2(x, x0, x1);
        const F2 phi = f2(x0 > 0.0f ? 1.0f - h0 : h0, x1 > 0.0f ? 1.0f - h1 : h1);
        return fma2(x * f2(0.39894228040143268f), g, phi);
    } else if constexpr (ACT == kActGeluTanh) {
        const F2 c = f2(-1.5957691216057308f * kLog2e), x2 = x * x;
        const F2 s = rcp_2(exp2_2(x * fma2(c * f2(0.044715f), x2, c)) + f2(1.0f));
        const F2 d = fma2(f2(1.5957691216057308f * 3.0f * 0.044715f), x2, f2(1.5957691216057308f));
        return fma2(x * s * fma2(s, f2(-1.0f), f2(1.0f)), d, s);
    } else if constexpr (ACT == kActSilu) {
        const F2 s = rcp_2(exp2_2(x * f2(-kLog2e)) + f2(1.0f));
        return s * fma2(x, fma2(s, f2(-1.0f), f2(1.0f)), f2(1.0f));
    } else {
        return f2(1.0f);
    }
}

__device__ __forceinline__ float load16(const void *p, int64_t i, int bf16)
{
    const uint16_t u = static_cast<const uint16_t *>(p)[i];
    return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                : __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ uint16_t round16(float v, int bf16)
{
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

template <int OUT>
__device__ __forceinline__ float load_as(const void *p, int64_t i)
{
    if constexpr (OUT == kOutF32)
        return static_cast<const float *>(p)[i];
    else
        return load16(p, i, OUT == kOutBF16);
}

template <int OUT>
__device__ __forceinline__ void store_as(void *p, int64_t i, float v)
{
    if constexpr (OUT == kOutF32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = round16(v, OUT == kOutBF16);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16)
{
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4 &v, float (&x)[8])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            x[2 * k] = __uint_as_float(u[k] << 16);
            x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[k]));
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
}

// Range of group g, clamped into the `tokens` that exist whatever the offsets say.
__device__ __forceinline__ void group_range(const int64_t *offsets, int tokens, int g, int &begin,
                                            int &end)
{
    if (!offsets) {
        begin = 0;
        end = tokens;
        return;
    }
    const int64_t b = offsets[g], e = offsets[g + 1], c = tokens;
    begin = static_cast<int>(b < 0 ? 0 : (b > c ? c : b));
    end = static_cast<int>(e < begin ? begin : (e > c ? c : e));
}

// What exponentials are taken relative to: the maximum so far, or zero where that is -inf
// (nothing but -inf).  exp(x - base) subtracts before it scales by log2 e: x = base gives
// exactly 1, however often a sum is rescaled, where x log2 e less the rounded base log2 e
// would give 1 + that rounding each time (100003 logits up to 103: lse off by 5.4e-4 so, under
// 1.6e-5 as it is).
__device__ __forceinline__ float exp_base(float mx) { return mx == -INFINITY ? 0.0f : mx; }
__device__ __forceinline__ float exp_from(float x, float base) { return exp2_fast((x - base) * kLog2e); }
__device__ __forceinline__ F2 exp_from(F2 x, F2 minus_base) { return exp2_2((x + minus_base) * f2(kLog2e)); }

// (maximum, sum of exponentials relative to it) of two sets of logits together.
__device__ __forceinline__ float2 join_stats(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x), base = exp_base(m);
    return make_float2(m, a.y * exp_from(a.x, base) + b.y * exp_from(b.x, base));
}

// Launch with programmatic stream serialization: the kernel waits in griddepcontrol.wait
// before it reads anything, so a chain of the library's kernels hides each launch.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t s, size_t smem,
                       Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tcg
