// GELU (erf) into bf16 from a table in LDS, for the epilogue of large tiles of 8-bit operands:
// v Phi(v) = max(v, 0) - t Phi(-t), t = |v|, with Phi(-t) linear in each interval of h =
// 1 / 256.  A line that is as wrong at its ends as in its middle is off by h^2 t phi(t) / 16,
// which is 2.4e-7 at most, and of Phi(-t) itself about h^2 t^2 / 16: the result is right to
// 4.9 u |v|, u = 2^-24, and to 1.8e-4 of itself down to -12.9 (gelu_erf: 8.1 u |v| and 1.6e-4;
// a bf16 rounding: 3.9e-3).  Below it ends in 0.
//
// Six vector instructions and a read of 8 bytes a value, which runs beside them, for 13 and an
// exponential.  25728 x 1024 -> 4096 with bias: 145 us, with gelu_erf 168, without an activation 132;
// gated 16384 x 4096 -> 14336 1406 and 1448.
#pragma once

#include "ffn_tile.h"

namespace dyra {

struct GeluTable {
    static constexpr int STEPS = 256;                       // lines of 1
    static constexpr int N = 27 * 128, LAST = 3379;         // whole KB; from 13.2 on the lines are 0
    float line[N][2];                                       // Phi(-t) = line[0] + line[1] t
};
// Mills' ratio m = Phi(-t) / phi(t) by Taylor steps down from the last line (m' = t m - 1, and
// m^(n+1) = t m^(n) + n m^(n-1)), a direction in which errors fade.
constexpr GeluTable gelu_table() {
    GeluTable r{};
    // Line i serves what rounds to it in eighths: [i - 1/16, i + 15/16) h.
    const double h = 1.0 / GeluTable::STEPS;
    double t = (GeluTable::LAST - 1.0 / 16) * h, m = 0, phi = 5.902728632586625e-39;  // phi of it
    for (int k = 60; k > 0; --k) m = k / (t + m);  // the continued fraction of Mills' ratio
    m = 1 / (t + m);
    double f = m * phi;
    for (int i = GeluTable::LAST - 1; i >= 0; --i) {
        double d0 = m, d1 = t * m - 1, step = -h, low = m + step * d1;
        for (int n = 1; n < 7; ++n) {
            const double d2 = t * d1 + n * d0;
            step *= -h / (n + 1);
            low += step * d2;
            d0 = d1;
            d1 = d2;
        }
        const double x = h * (t - h / 2);  // phi(t - h) = phi(t) exp(x)
        double e = 1;
        for (int n = 8; n > 0; --n) e = 1 + e * x / n;
        phi *= e;
        t -= h;
        const double g = low * phi, slope = (f - g) / h;
        const double off = 1 - h * h * (t + h / 2) / (8 * (m + low));
        r.line[i][0] = (float)((g - slope * t) * off);
        r.line[i][1] = (float)(slope * off);
        m = low;
        f = g;
    }
    return r;
}
static __device__ constexpr GeluTable kGeluTable = gelu_table();

// Wavefront `wave` of 8 copies its part into `table`.
__device__ __forceinline__ void copy_gelu_table(char *table, int wave, int lane) {
    const __amdgpu_buffer_rsrc_t from = panel(&kGeluTable, sizeof(GeluTable));
    for (int block = wave; block < (int)sizeof(GeluTable) / 1024; block += 8)
        buffer_to_lds16(from, (uint32_t)(1024 * block + 16 * lane), 0, table + 1024 * block);
}
// v to gelu(v), the reads of G values in flight together.  `table` is aligned to 8 bytes.
template <int G, int C> __device__ __forceinline__ void gelu_from(const char *table, float (&v)[C]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef const __attribute__((address_space(3))) f32x2 *Line;
    // A float32 from 4096 on has a last place of 2^-11 = h / 8: the low bits of 4096 + t +
    // address / 2048 are the table's address and t in eighths of a line.
    const unsigned base = (unsigned)(size_t)(const __attribute__((address_space(3))) char *)table;
    const float magic = __uint_as_float(0x45800000u + base);
#pragma unroll
    for (int p = 0; p < C; p += G) {
        float t[G];
        f32x2 line[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
            t[q] = __builtin_amdgcn_fmed3f(fabsf(v[p + q]), 0.f, (float)GeluTable::LAST / GeluTable::STEPS);  // of NaN 0
            line[q] = *(Line)(size_t)(__float_as_uint(t[q] + magic) & 0x3fff8u);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < G; ++q)  // NaN stays NaN
            v[p + q] = __builtin_fmaf(-t[q], __builtin_fmaf(line[q][1], t[q], line[q][0]), __builtin_elementwise_maximum(v[p + q], 0.f));
    }
}

}  // namespace dyra
