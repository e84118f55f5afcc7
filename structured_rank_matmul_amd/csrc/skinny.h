// Products of a few tokens with streamed weights, for the feed-forward kernels
// of few tokens (skinny.hip, moe.hip): a wavefront multiplies 16 weight rows of
// MATS matrices with 16 TN tokens over a range of K.  The weights and the
// tokens are read from global memory in fragment form (16 bytes of one row per
// lane), UNROLL steps of 32 requested at once; every load is unconditional
// (rows and steps past the end are clamped by the caller or the step count, a
// last partial step is read through a zero chunk).
#pragma once

#include "ffn_tile.h"

namespace dyra {

__device__ __align__(16) static const unsigned g_skinny_zero[4] = {0, 0, 0, 0};

// This lane's 8 elements of a 32-deep step: p points at element 8 (lane / 16)
// of the step and `left` elements of the row are left from there on.
__device__ __forceinline__ bf16x8 step_frag(const bf16 *p) { return *reinterpret_cast<const bf16x8 *>(p); }
__device__ __forceinline__ f32x8 step_frag(const float *p) { return ld_frag(p); }
__device__ __forceinline__ bf16x8 step_frag_tail(const bf16 *p, int64_t left) {
    return *reinterpret_cast<const bf16x8 *>(left > 0 ? (const void *)p : (const void *)g_skinny_zero);
}
__device__ __forceinline__ f32x8 step_frag_tail(const float *p, int64_t left) {
    const f32x4 lo = *reinterpret_cast<const f32x4 *>(left > 0 ? (const void *)p : (const void *)g_skinny_zero);
    const f32x4 hi = *reinterpret_cast<const f32x4 *>(left > 4 ? (const void *)(p + 4) : (const void *)g_skinny_zero);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// acc[m][t] += W_m[16 rows] X_t[16 tokens]^T over steps [s0, s1) of 32.
// w[m], x[t]: this lane's row pointers, already at element 8 (lane / 16).
template <typename E, int MATS, int TN, int UNROLL>
__device__ __forceinline__ void skinny_product(const E *const (&w)[MATS], const E *const (&x)[TN], int64_t K, int s0,
                                               int s1, f32x4 (&acc)[MATS][TN]) {
    typedef typename Frag<E>::type F;
    const int g = (threadIdx.x & 63) >> 4;
    const int whole = (int)(K / 32);  // steps with every element
    int s = s0;
    const int e = s1 < whole ? s1 : whole;
    for (; s + UNROLL <= e; s += UNROLL) {
        F fw[UNROLL][MATS], fx[UNROLL][TN];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
            for (int m = 0; m < MATS; ++m) fw[u][m] = step_frag(w[m] + (int64_t)(s + u) * 32);
#pragma unroll
            for (int t = 0; t < TN; ++t) fx[u][t] = step_frag(x[t] + (int64_t)(s + u) * 32);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int t = 0; t < TN; ++t) acc[m][t] = mma32(acc[m][t], fw[u][m], fx[u][t]);
    }
    for (; s < s1; ++s) {
        const int64_t left = K - (int64_t)s * 32 - 8 * g;
        F fw[MATS], fx[TN];
#pragma unroll
        for (int m = 0; m < MATS; ++m) fw[m] = step_frag_tail(w[m] + (int64_t)s * 32, left);
#pragma unroll
        for (int t = 0; t < TN; ++t) fx[t] = step_frag_tail(x[t] + (int64_t)s * 32, left);
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int t = 0; t < TN; ++t) acc[m][t] = mma32(acc[m][t], fw[m], fx[t]);
    }
}

}  // namespace dyra
