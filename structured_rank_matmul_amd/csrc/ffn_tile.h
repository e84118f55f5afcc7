// Device building blocks shared by the feed-forward kernels: 16 x 16 MFMA
// blocks 32 deep, activations, guarded 16-byte loads.
//
// Operands of one 16 x 16 block: lane l holds 8 contraction elements
// k = 8 (l / 16) .. + 7 of row (first operand) or column (second operand)
// l % 16.  For bf16 that is one v_mfma_f32_16x16x32_bf16; for float32 the same
// 8 elements feed eight v_mfma_f32_16x16x4_f32 steps, step t contracting
// element t of every lane group, the same permutation of k for both operands.
// Result (both): lane l holds column l % 16, register t row 4 (l / 16) + t.
// The weights are always the first operand, so a lane's four registers are
// four consecutive output features of one token.
#pragma once

#include "ffn_kernels.h"
#include "mfma_tile.h"

#include <type_traits>

namespace dyra {

__device__ __forceinline__ f32x4 mma32(f32x4 acc, bf16x8 a, bf16x8 b) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma32(f32x4 acc, f32x8 a, f32x8 b) {
#pragma unroll
    for (int t = 0; t < 8; ++t) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[t], b[t], acc, 0, 0, 0);
    return acc;
}

// exp(v) and 1 / v by the hardware's exp2 and reciprocal (1 ulp each; the
// product with log2(e) adds |v| u to the exponent's error).  The compiler's own
// expf and division take about ten instructions each: at 25728 x 4096 outputs
// a SiLU epilogue cost 24 us with them.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896341f); }
__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }

// Phi(v) = (1 + erf(v / sqrt 2)) / 2 by Abramowitz and Stegun 7.1.26: with
// x = |v| / sqrt 2, t = 1 / (1 + p x), 1 - erf(x) = (a1 t + .. + a5 t^5) e^{-x^2},
// off by at most 1.5e-7, so v Phi(v) by 0.75e-7 |v|.  The library's erff costs
// three times as many instructions (117 us at 25728 x 4096 outputs).
__device__ __forceinline__ float normal_cdf(float v) {
    const float t = fast_rcp(1.f + 0.23164189f * fabsf(v));
    const float poly = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    const float tail = 0.5f * poly * __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
    return v >= 0.f ? 1.f - tail : tail;
}

// act(v) in float32, within a few u |v| (u = 2^-24).  gelu is the exact form
// v Phi(v); gelu_tanh's v/2 (1 + tanh(w)) is v / (1 + exp(-2 w)).  PRECISE
// (float32 outputs) takes erf from the device library.
template <bool PRECISE, int C> __device__ __forceinline__ void activate(float (&v)[C], int act) {
    if (act == kActRelu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] = v[q] < 0.f ? 0.f : v[q];  // NaN stays
    } else if (act == kActGelu) {
#pragma unroll
        for (int q = 0; q < C; ++q)
            v[q] *= PRECISE ? 0.5f * (1.f + erff(v[q] * 0.70710678118654752f)) : normal_cdf(v[q]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int q = 0; q < C; ++q) {
            const float w = 0.79788456080286536f * (v[q] + 0.044715f * v[q] * v[q] * v[q]);
            v[q] *= fast_rcp(1.f + fast_exp(-2.f * w));
        }
    } else if (act == kActSilu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] *= fast_rcp(1.f + fast_exp(-v[q]));
    }
}

// N consecutive elements as float32 (16-byte accesses where `vec`; only the
// first `have` exist).
template <typename T, int N> __device__ __forceinline__ void load_row(const T *p, float (&v)[N], bool vec, int have) {
    constexpr int V = 16 / (int)sizeof(T);
    static_assert(N % V == 0, "whole 16-byte chunks");
    if (vec && have >= N) {
#pragma unroll
        for (int q = 0; q < N; q += V) {
            union { u32x4 u; T e[V]; } w;
            w.u = *reinterpret_cast<const u32x4 *>(p + q);
#pragma unroll
            for (int i = 0; i < V; ++i) v[q + i] = to_f32(w.e[i]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = q < have ? to_f32(p[q]) : 0.f;
    }
}
template <typename T, int N> __device__ __forceinline__ void store_row(T *p, const float (&v)[N], bool vec, int have) {
    constexpr int V = 16 / (int)sizeof(T);
    if (vec && have >= N) {
#pragma unroll
        for (int q = 0; q < N; q += V) {
            union { u32x4 u; T e[V]; } w;
#pragma unroll
            for (int i = 0; i < V; ++i) w.e[i] = to_elem<T>(v[q + i]);
            *reinterpret_cast<u32x4 *>(p + q) = w.u;
        }
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (q < have) p[q] = to_elem<T>(v[q]);
    }
}

}  // namespace dyra
