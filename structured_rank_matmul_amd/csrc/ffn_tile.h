// Device building blocks shared by the feed-forward kernels: 16 x 16 MFMA
// blocks 32 deep, activations, guarded 16-byte loads.
//
// Operands of one 16 x 16 block: lane l holds 8 contraction elements of row
// (first operand) or column (second operand) l % 16.  For bf16 these are k = 8 (l / 16)
// .. + 7 of one v_mfma_f32_16x16x32_bf16.  For float32 they are k = 4 (l / 16) .. + 3
// and 16 more of the same, and feed eight v_mfma_f32_16x16x4_f32 steps, step t
// contracting element t of every lane group, the same permutation of k for both
// operands.  (Chunks of 16 bytes g and 4 + g of a slab, as bf16 reads in its two steps: 2 g
// and 2 g + 1 would meet on a bank under the same swizzle.)
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

// A buffer resource over `bytes` (at most 2 GiB) from `p` on; loads past them, at
// kOutside among them, give 0.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t panel(const void *p, int64_t bytes = kOutside - 1) {
    const int n = bytes < (int64_t)kOutside - 1 ? (int)bytes : (int)(kOutside - 1);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, n, 0x00027000);
}
__device__ __forceinline__ void buffer_to_lds16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, char *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, (int)voff, (int)soff, 0, 0);
}
template <int N> __device__ __forceinline__ void wait_lds_and_vm() {
    // lgkmcnt(0) and vmcnt(N): gfx9 encoding, expcnt left at its maximum
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// exp(v) and 1 / v by the hardware's exp2 and reciprocal (1 ulp each; the
// product with log2(e) adds |v| u to the exponent's error).  The compiler's own
// expf and division take about ten instructions each: at 25728 x 4096 outputs
// a SiLU epilogue cost 24 us with them.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896341f); }
__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }

// exp(-v) to 4 u (u = 2^-24), in [2^-128, 2^128]: 2^-h for h = v log2(e) rounded, times
// 1 - r ln 2 for what the rounding left out.  Float32, 12608 x 768
// -> 3000 with silu: 475 us with fast_exp, 479 with this, 496 with the compiler's expf
// and division.
__device__ __forceinline__ float exp_minus(float v) {
    const float t = fminf(fmaxf(v, -88.5f), 88.5f), h = t * 1.44269504088896341f;
    const float r = __builtin_fmaf(t, 1.92596299e-8f, __builtin_fmaf(t, 1.44269504088896341f, -h));
    const float e = __builtin_amdgcn_exp2f(-h);
    return __builtin_fmaf(e, r * -0.693147181f, e);
}

// v Phi(v) = v (1 + erf(v / sqrt 2)) / 2 for results in bf16, as max(v, 0) - t Phi(-t)
// with t = |v| and Phi(-t) = 2^-P(t).  P is a least-maximum fit (own) to -log2 Phi(-t):
// where 2^-P(t) is a normal float32 (t <= 13.2) its error may be 1e-4 of Phi(-t) or
// 3e-7, whichever is less; past 14.5 it is 0.  With float32 evaluation the result is
// right to 1.6e-4 of itself (a bf16 rounding: 3.9e-3) and to 8.1 u |v|, u = 2^-24,
// over a dense grid of |v| <= 12.9; below that it ends in 0, its limit.  NaN stays NaN.  A fit to
// the absolute error alone, v / (1 + 2^(v Q(v^2))), was 7 % off at v = -4.5 and 70 % at
// -5.  ViT-L fc1, 25728 x 1024 -> 4096: 225 us; with that fit 222, with degree 8 here
// (6e-4) 219, with 11 230, without an activation 192.
__device__ __forceinline__ float gelu_erf(float v) {
    const float t = __builtin_elementwise_minimum(fabsf(v), 14.5f);
    float p = 2.506931329e-10f;
    p = __builtin_fmaf(p, t, -1.331301647e-08f);
    p = __builtin_fmaf(p, t, 2.455076356e-07f);
    p = __builtin_fmaf(p, t, -7.569577178e-07f);
    p = __builtin_fmaf(p, t, -4.255376189e-05f);
    p = __builtin_fmaf(p, t, 8.341055363e-04f);
    p = __builtin_fmaf(p, t, -8.210643195e-03f);
    p = __builtin_fmaf(p, t, 5.347734690e-02f);
    p = __builtin_fmaf(p, t, 4.588192701e-01f);
    p = __builtin_fmaf(p, t, 1.151160121e+00f);
    p = __builtin_fmaf(p, t, 9.999988079e-01f);
    return __builtin_fmaf(-t, __builtin_amdgcn_exp2f(-p), __builtin_elementwise_maximum(v, 0.f));
}

// act(v) in float32, within a few u |v| (u = 2^-24).  gelu is the exact form
// v Phi(v); gelu_tanh's v/2 (1 + tanh(w)) is v / (1 + exp(-2 w)).  PRECISE
// (float32 outputs) takes erfc from the device library: v/2 erfc(-v / sqrt 2), as
// 1 + erf cancels for v < 0 (3 % of the result at v = -5); and silu's exponential with the
// rounding of its argument put right, which is |v| u of a small result.
template <bool PRECISE, int C> __device__ __forceinline__ void activate(float (&v)[C], int act) {
    if (act == kActRelu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] = v[q] < 0.f ? 0.f : v[q];  // NaN stays
    } else if (act == kActGelu) {
#pragma unroll
        for (int q = 0; q < C; ++q)
            v[q] = PRECISE ? v[q] * (0.5f * erfcf(v[q] * -0.70710678118654752f)) : gelu_erf(v[q]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int q = 0; q < C; ++q) {
            // exp(-2 w) = 2^(v (a + b v^2)): a = -2 sqrt(2 / pi) log2(e), b = 0.044715 a
            const float e = v[q] * (-2.3022082f + -0.10294324f * (v[q] * v[q]));
            v[q] *= fast_rcp(1.f + __builtin_amdgcn_exp2f(e));
        }
    } else if (act == kActSilu) {
#pragma unroll
        for (int q = 0; q < C; ++q) v[q] *= fast_rcp(1.f + (PRECISE ? exp_minus(v[q]) : fast_exp(-v[q])));
    }
}

// N consecutive elements as float32, of which the first `have` exist: 16-byte
// accesses of any alignment where all do (gfx950 takes them; rows of odd length
// stored by elements cost an epilogue of 1501 x 1003 floats 6 us of 14).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T, int N> __device__ __forceinline__ void load_row(const T *p, float (&v)[N], int have) {
    constexpr int V = 16 / (int)sizeof(T);
    static_assert(N % V == 0, "whole 16-byte chunks");
    if (have >= N) {
#pragma unroll
        for (int q = 0; q < N; q += V) {
            union { u32x4 u; T e[V]; } w;
            w.u = *reinterpret_cast<const u32x4_any *>(p + q);
#pragma unroll
            for (int i = 0; i < V; ++i) v[q + i] = to_f32(w.e[i]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = q < have ? to_f32(p[q]) : 0.f;
    }
}
// Eight elements of a residual row in flight: requested for a batch of rows before
// the first is used (loads used one by one cost each its latency).
template <typename T> struct Residual8 {
    u32x4 c[8 * (int)sizeof(T) / 16];
    __device__ __forceinline__ void request(const T *p) {
#pragma unroll
        for (int q = 0; q < 8 * (int)sizeof(T) / 16; ++q) c[q] = *reinterpret_cast<const u32x4_any *>((const char *)p + 16 * q);
    }
    __device__ __forceinline__ void add_to(float (&v)[8]) const {
        union { u32x4 u[8 * sizeof(T) / 16]; T e[8]; } w;
#pragma unroll
        for (int q = 0; q < 8 * (int)sizeof(T) / 16; ++q) w.u[q] = c[q];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += to_f32(w.e[q]);
    }
};
// The same of a row of which the first `have` (0 .. 8) exist; columns past them
// repeat the last one and are not stored.
template <typename T> __device__ __forceinline__ void add_row(float (&v)[8], const T *p, int have) {
    if (have >= 8) {
        Residual8<T> r;
        r.request(p);
        r.add_to(v);
    } else if (have > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += to_f32(p[q < have ? q : have - 1]);
    }
}
// Eight results of a row, of which the first `have` (0 .. 8) exist: a 16-byte store (two
// for float32), or, in the last columns, one each of four, two and one element.
__device__ __forceinline__ void store_row(float *p, const float (&v)[8], int have) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef f32x4 f32x4_any __attribute__((aligned(4)));
    typedef f32x2 f32x2_any __attribute__((aligned(4)));
    const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    const bool four = have & 4, two = have & 2;
    if (have >= 8 || four) *reinterpret_cast<f32x4_any *>(p) = lo;
    if (have >= 8) {
        *reinterpret_cast<f32x4_any *>(p + 4) = hi;
        return;
    }
    const f32x4 rest = four ? hi : lo;
    if (two) *reinterpret_cast<f32x2_any *>(p + (have & 4)) = f32x2{rest[0], rest[1]};
    if (have & 1) p[have & 6] = two ? rest[2] : rest[0];
}
__device__ __forceinline__ void store_row(bf16 *p, const float (&v)[8], int have) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    typedef u32x2 u32x2_any __attribute__((aligned(2)));
    typedef unsigned u32_any __attribute__((aligned(2)));
    union { u32x4 u; bf16 e[8]; } w;
#pragma unroll
    for (int q = 0; q < 8; ++q) w.e[q] = to_elem<bf16>(v[q]);
    if (have >= 8) {
        *reinterpret_cast<u32x4_any *>(p) = w.u;
        return;
    }
    const bool four = have & 4, two = have & 2;
    if (four) *reinterpret_cast<u32x2_any *>(p) = u32x2{w.u[0], w.u[1]};
    if (two) *reinterpret_cast<u32_any *>(p + (have & 4)) = four ? w.u[2] : w.u[0];
    const unsigned last = four ? (two ? w.u[3] : w.u[2]) : (two ? w.u[1] : w.u[0]);
    if (have & 1) *reinterpret_cast<unsigned short *>(p + (have & 6)) = (unsigned short)last;
}

}  // namespace dyra
