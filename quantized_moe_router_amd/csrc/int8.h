// Device helpers shared by the INT8 W8A16 linear layer's kernels.
#pragma once

#include "common.h"

namespace moe {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Stored bytes 2i and 2i+1 of a word -> fp16 pair (q - 128), exact.  The
// permute takes result bytes from {0x64646464 (bytes 4-7), w (bytes 0-3)}.
template <int I>
__device__ __forceinline__ h2_t code_pair(uint32_t w)
{
    constexpr uint32_t sel = I == 0 ? 0x04010400u : 0x04030402u;
    const uint32_t p = __builtin_amdgcn_perm(0x64646464u, w, sel);
    return __builtin_bit_cast(h2_t, p) + h2_t{(_Float16)-1152.f, (_Float16)-1152.f};
}

// 8 bf16 (natural order) -> 8 fp16 (natural order); exact in fp16's normal
// range, toward zero outside it (saturating at 65504).
__device__ __forceinline__ u32x4_t bf16x8_to_f16x8(u32x4_t v)
{
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(bf16_lo(v[j]), bf16_hi(v[j])));
    return o;
}

// ---------------------------------------------------------------------------
// Epilogue of the fused variant (F = true in the kernels below):
//   out[t][r] = rnd(residual[t][r] + act(sum + bias[r]))
// in fp32, one rounding.  Everything happens on the sum in registers, so the
// activation and the addition cost no pass over [T][N] of their own.
// The activations are accurate to a few units of fp32's last place (an fp32
// output shows errors that a bf16 one would hide), but for the far negative
// tails of GELU and its tanh form: there the rounding of the argument of erfc
// or the exponential moves the result by up to v^2 or 10 |u| units.
// ---------------------------------------------------------------------------
// 1 / (1 + e^-z), as t / (1 + t) or 1 / (1 + t) with t = e^-|z| in (0, 1]: no
// overflow, and a divisor in [1, 2], whose reciprocal is the hardware's with
// one Newton step.  t is 2^h (1 + r ln 2) with h = fp32(-|z| log2 e) and r what
// h leaves of the product (the hardware's exponential alone, on the rounded
// product, is off by |z| units of the last place).  Half the instructions of
// expf and a division: 512 tokens of a [10240, 320] layer with SiLU and a
// residual 18.7 us against 20.2, 2048 of [4096, 2560] 73.8 against 74.9.
// Below fp32's normal range t is zero.
__device__ __forceinline__ float sigmoid(float z)
{
    constexpr float kL = 1.44269504088896341f;           // log2 e as fp32, and the rest of it
    constexpr float kLr = (float)(1.44269504088896340736 - (double)kL);
    const float a = -fabsf(z), h = a * kL;
    const float r = fmaf(a, kL, -h) + a * kLr;
    float t = __builtin_amdgcn_exp2f(h);
    t = h < -126.f ? 0.f : fmaf(t * 0.69314718055994531f, r, t);   // -inf, too, whose r is not a number
    const float d = 1.f + t;
    float q = __builtin_amdgcn_rcpf(d);
    q = fmaf(fmaf(-d, q, 1.f), q, q);
    return z < 0.f ? t * q : q;   // a NaN passes through t
}

// One body for the three that hold a sigmoid: kernels of a few microseconds
// fetch their code anew at every launch, and a copy of every activation per
// output cost the short-K kernel more than its products.
__device__ __forceinline__ float activate(float v, int kind)   // kind is uniform over the launch
{
    if (kind == kActNone) return v;
    if (kind == kActRelu) return v < 0.f ? 0.f : v;   // a NaN passes
    if (kind == kActGelu) return 0.5f * v * erfcf(-0.70710678118654752f * v);
    float z = v;
    // 0.5 (1 + tanh u) = sigmoid(2 u), without tanh's cancellation near -1
    if (kind == kActGeluTanh) z = 2.f * 0.79788456080286536f * fmaf(0.044715f * v * v, v, v);
    return (kind == kActSigmoid ? 1.f : v) * sigmoid(z);
}

__device__ __forceinline__ void finish(const Int8Epilogue &e, int t, int r, float v)
{
    if (e.bias) v += load_typed(e.bias, e.bias_type, r);
    v = activate(v, e.activation);
    if (e.residual) v += load_typed(e.residual, e.residual_type, t * e.residual_stride + r);
    store_typed(e.out, e.out_type, t * e.out_stride + r, v);
}

// Columns r .. r + 3 of one row (r a multiple of 4, e.vec set).
__device__ __forceinline__ void finish4(const Int8Epilogue &e, int t, int r, float4 v)
{
    if (e.bias) {
        const float4 b = load_typed4(e.bias, e.bias_type, r);
        v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
    }
    if (e.activation != kActNone)
        v = make_float4(activate(v.x, e.activation), activate(v.y, e.activation), activate(v.z, e.activation),
                        activate(v.w, e.activation));
    if (e.residual) {
        const float4 b = load_typed4(e.residual, e.residual_type, t * e.residual_stride + r);
        v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
    }
    store_typed4(e.out, e.out_type, t * e.out_stride + r, v);
}

// Column r of rows t, t + step, .. (four, those below T), with its bias: for
// outputs whose columns share no aligned word.  The residual is asked for
// first, so that its four loads are waited for once.
__device__ __forceinline__ void finish_rows(const Int8Epilogue &e, int t, int step, int T, int r, float bias,
                                            const float (&v)[4])
{
    float res[4] = {0.f, 0.f, 0.f, 0.f};
    if (e.residual) {
        size_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = min(t + i * step, T - 1) * e.residual_stride + r;
        if (e.residual_type == kF32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) res[i] = static_cast<const float *>(e.residual)[at[i]];
        } else {
            uint16_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = static_cast<const uint16_t *>(e.residual)[at[i]];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                res[i] = e.residual_type == kBf16 ? bf16_to_f32(b[i]) : (float)__builtin_bit_cast(_Float16, b[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t + i * step < T)
            store_typed(e.out, e.out_type, (t + i * step) * e.out_stride + r, activate(v[i] + bias, e.activation) + res[i]);
}

// Columns r .. r + 3 of rows t, t + step, .. (four, those below T), bias and
// activation taken in already, r a multiple of 4 and e.vec set: the residual's
// four loads are waited for once.
__device__ __forceinline__ void finish_rows4(const Int8Epilogue &e, int t, int step, int T, int r, float4 (&v)[4])
{
    if (e.residual) {
        float4 res[4];
        if (e.residual_type == kF32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                res[i] = load_typed4(e.residual, kF32, min(t + i * step, T - 1) * e.residual_stride + r);
        } else if (e.residual_type == kBf16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                res[i] = load_typed4(e.residual, kBf16, min(t + i * step, T - 1) * e.residual_stride + r);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                res[i] = load_typed4(e.residual, kF16, min(t + i * step, T - 1) * e.residual_stride + r);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = make_float4(v[i].x + res[i].x, v[i].y + res[i].y, v[i].z + res[i].z, v[i].w + res[i].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t + i * step < T) store_typed4(e.out, e.out_type, (t + i * step) * e.out_stride + r, v[i]);
}

}  // namespace moe
