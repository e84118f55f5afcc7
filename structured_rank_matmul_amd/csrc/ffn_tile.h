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

// act(v) in float32.  gelu is the exact form 0.5 v (1 + erf(v / sqrt 2));
// gelu_tanh's 0.5 v (1 + tanh(u)) is v / (1 + exp(-2 u)).
template <int C> __device__ __forceinline__ void activate(float (&v)[C], int act) {
    if (act == kActRelu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] = v[q] > 0.f ? v[q] : (v[q] != v[q] ? v[q] : 0.f);
    } else if (act == kActGelu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] = 0.5f * v[q] * (1.f + erff(v[q] * 0.70710678118654752f));
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int q = 0; q < C; ++q) {
            const float u = 0.79788456080286536f * (v[q] + 0.044715f * v[q] * v[q] * v[q]);
            v[q] = v[q] / (1.f + expf(-2.f * u));
        }
    } else if (act == kActSilu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] = v[q] / (1.f + expf(-v[q]));
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
