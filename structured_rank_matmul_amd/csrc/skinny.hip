// Linear layer and gated pair for few tokens, bound by reading the weights once.
//
// A workgroup takes units of 16 weight rows (16 output features, or 8 gate and
// the same 8 up rows) and streams them through its wavefronts' rings (skinny.h);
// a unit's epilogue runs while the next unit's slabs are landing.  More than 16
// TB tokens are taken in groups, one after the other on the same unit.
//
// 16 tokens, gated 4096 -> 14336 (235 MB of weights): see kSkinnyTokens in
// ffn_api.hip for what the other kernel takes.
#include "skinny.h"

#include <algorithm>

namespace dyra {

namespace {

template <typename E, typename O, bool GATED, int TB> struct UnitPositions {
    static constexpr int R = GATED ? 8 : 16;            // output features of a unit
    static constexpr int kFinishers = 16 * R * TB;
    const LinearArgs<E, O> &a;
    int units, groups, count;
    __device__ UnitPositions(const LinearArgs<E, O> &args, int n, int g) : a(args), units(n), groups(g) {
        count = (n - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * g;
    }
    __device__ __forceinline__ int unit(int p) const { return (int)blockIdx.x + p / groups * (int)gridDim.x; }
    __device__ __forceinline__ int64_t token0(int p) const { return 16 * TB * (int64_t)(p % groups); }
    __device__ __forceinline__ void weights(int p, SlabRows &w) const {
        const int64_t f0 = (int64_t)unit(p) * R;
        const uint32_t ld = (uint32_t)(a.ldw * sizeof(E));
        const int last = (int)min((int64_t)R, a.N - f0) - 1;  // rows past the end repeat the last one
        w.buf[0] = panel(a.W0 + f0 * a.ldw);
        w.buf[1] = GATED ? panel(a.W1 + f0 * a.ldw) : w.buf[0];
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w.off[q] = (uint32_t)min(GATED ? slab_row(q) & 7 : slab_row(q), last) * ld + slab_chunk(q);
    }
    __device__ __forceinline__ bool new_tokens(int p) const { return p == 0 || groups > 1; }
    __device__ __forceinline__ int blocks(int p) const { return TB == 2 && a.M - token0(p) > 16 ? 2 : 1; }
    __device__ __forceinline__ void tokens(int p, SlabRows (&x)[TB]) const {
        const int64_t t0 = token0(p);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            x[t].buf[0] = x[t].buf[1] = panel(a.X + t0 * a.ldx);
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // rows past the end read nothing
                const int r = 16 * t + slab_row(q);
                x[t].off[q] = t0 + r < a.M ? (uint32_t)r * (uint32_t)(a.ldx * sizeof(E)) + slab_chunk(q) : kOutside;
            }
        }
    }
    __device__ __forceinline__ void finish(int p, const float *sums, int thread) const {
        const int f = thread % R, t = thread / R;
        const int64_t tok = token0(p) + t, c = (int64_t)unit(p) * R + f;
        if (t >= 16 * TB || tok >= a.M || c >= a.N) return;
        const float *block = sums + (t >> 4) * kWaves * kBlockSums;
        float y[1] = {joined(block, t & 15, f) + (a.b0 ? to_f32(a.b0[c]) : 0.f)};
        activate<sizeof(O) == 4>(y, a.act);
        if constexpr (GATED) y[0] *= joined(block, t & 15, 8 + f) + (a.b1 ? to_f32(a.b1[c]) : 0.f);
        else if (a.R) y[0] += to_f32(a.R[tok * a.ldr + c]);
        a.Y[tok * a.ldy + c] = to_elem<O>(y[0]);
    }
};

template <typename E, typename O, bool GATED, int SLABS, int TB>
__global__ __launch_bounds__(kThreads) void skinny_kernel(LinearArgs<E, O> a, int units, int groups) {
    __shared__ __align__(16) StreamLds<TB> lds;
    const UnitPositions<E, O, GATED, TB> positions(a, units, groups);
    stream_products<E, SLABS, TB>(positions, (int)(a.K * (int)sizeof(E)), lds);
}

template <typename E, typename O, bool GATED, int SLABS, int TB>
hipError_t launch_slabs(const LinearArgs<E, O> &a, hipStream_t st) {
    const int units = (int)((a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16));
    const int groups = (int)((a.M + 16 * TB - 1) / (16 * TB));
    // at most one workgroup per CU, the same number of units each (224 x 4 units
    // rather than 128 x 4 and 128 x 3: 16 tokens, 4096 -> 14336, 29.4 -> 24.4 us)
    const int rounds = (units + 255) / 256;
    hipLaunchKernelGGL((skinny_kernel<E, O, GATED, SLABS, TB>), dim3((unsigned)((units + rounds - 1) / rounds)),
                       dim3(kThreads), 0, st, a, units, groups);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_skinny(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    // the smallest register space that holds a wavefront's slabs of the tokens
    // (8 registers a slab and block), or the largest that fits
    const int slabs = (int)((a.K * (int64_t)sizeof(E) + 128 * kWaves - 1) / (128 * kWaves));
    if (a.M <= 16) {
        if (slabs <= 2) return launch_slabs<E, O, GATED, 2, 1>(a, st);
        if (slabs <= 4) return launch_slabs<E, O, GATED, 4, 1>(a, st);
        if (slabs <= 8) return launch_slabs<E, O, GATED, 8, 1>(a, st);
        if (slabs <= 16) return launch_slabs<E, O, GATED, 16, 1>(a, st);
        return launch_slabs<E, O, GATED, 24, 1>(a, st);
    }
    if (slabs <= 4) return launch_slabs<E, O, GATED, 4, 2>(a, st);
    if (slabs <= 8) return launch_slabs<E, O, GATED, 8, 2>(a, st);
    return launch_slabs<E, O, GATED, 12, 2>(a, st);
}

template hipError_t launch_skinny<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_skinny<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_skinny<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
