// Linear layer and gated pair for few tokens, bound by reading the weights once.
//
// A workgroup takes units of 16 weight rows (16 output features, or 8 gate and
// the same 8 up rows); its eight wavefronts split K, each streaming its part
// through its own ring (skinny.h).  The ring runs on from unit to unit, so the
// sums of one unit meet in LDS, in a fixed order, and get their epilogue while
// the next unit's slabs are landing.
//
// A wavefront's part of K is the same in every unit, so where they fit its
// fragments of the tokens are loaded once and stay in registers (SLABS slabs,
// TB blocks of 16 tokens: 8 SLABS TB registers).  Where they do not, the
// tokens' slabs go through the ring beside the weights', in groups of 16 tokens
// on the same weights.  16 tokens, 4096 -> 14336 gated: 53.7 us with the tokens
// in the ring (they double what the copies move).
#include "lanes.h"
#include "skinny.h"

#include <algorithm>

namespace dyra {

namespace {

constexpr int kWaves = 8;
constexpr int kSumStride = 20;  // floats of a token's 16 sums, padded

template <typename E, typename O, bool GATED> struct Unit {
    static constexpr int R = GATED ? 8 : 16;  // output features
    static __device__ __forceinline__ void aim(const LinearArgs<E, O> &a, int unit, SlabRows &w) {
        const int64_t f0 = (int64_t)unit * R;
        const uint32_t ld = (uint32_t)(a.ldw * sizeof(E));
        const int last = (int)min((int64_t)R, a.N - f0) - 1;  // rows past the end repeat the last one
        w.buf[0] = panel(a.W0 + f0 * a.ldw);
        w.buf[1] = GATED ? panel(a.W1 + f0 * a.ldw) : w.buf[0];
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w.off[q] = (uint32_t)min(GATED ? slab_row(q) & 7 : slab_row(q), last) * ld + slab_chunk(q);
    }
    // Joins the wavefronts' sums of 16 tokens from t0 on, applies the epilogue and stores.
    static __device__ __forceinline__ void finish(const LinearArgs<E, O> &a, int unit, int64_t t0,
                                                  const float (*sums)[16 * kSumStride], int thread) {
        const int f = thread % R, t = thread / R;
        const int64_t tok = t0 + t, c = (int64_t)unit * R + f;
        if (t >= 16 || tok >= a.M || c >= a.N) return;
        float z[GATED ? 2 : 1] = {};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            z[0] += sums[v][t * kSumStride + f];
            if constexpr (GATED) z[1] += sums[v][t * kSumStride + 8 + f];
        }
        float y[1] = {z[0] + (a.b0 ? to_f32(a.b0[c]) : 0.f)};
        activate<sizeof(O) == 4>(y, a.act);
        if constexpr (GATED) y[0] *= z[1] + (a.b1 ? to_f32(a.b1[c]) : 0.f);
        else if (a.R) y[0] += to_f32(a.R[tok * a.ldr + c]);
        a.Y[tok * a.ldy + c] = to_elem<O>(y[0]);
    }
    static __device__ __forceinline__ void put(float *sums, const f32x4 &acc) {
        const int lane = threadIdx.x & 63;
        *reinterpret_cast<f32x4 *>(sums + (lane & 15) * kSumStride + 4 * (lane >> 4)) = acc;
    }
};

// This wavefront's slabs of K.
__device__ __forceinline__ void my_slabs(int row_bytes, int wave, int &s0, int &s1) {
    const int slabs = (row_bytes + 127) / 128, per = (slabs + kWaves - 1) / kWaves;
    s0 = min(slabs, wave * per);
    s1 = min(slabs, s0 + per);
}

// Tokens in registers: M <= 16 TB, at most SLABS slabs a wavefront.
template <typename E, typename O, bool GATED, int SLABS, int TB>
__global__ __launch_bounds__(64 * kWaves) void skinny_kernel(LinearArgs<E, O> a, int units) {
    using U = Unit<E, O, GATED>;
    __shared__ __align__(16) char ring_mem[kWaves * kRingBytes];
    __shared__ __align__(16) float sums[TB == 1 ? 2 : 1][TB][kWaves][16 * kSumStride];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row_bytes = (int)(a.K * (int)sizeof(E));
    int s0, s1;
    my_slabs(row_bytes, wave, s0, s1);

    // the stream of weights: slabs s0 .. s1 of unit after unit
    SlabRows w;
    SlabRing<E, false> ring{ring_mem + wave * kRingBytes};
    int in_unit = blockIdx.x, in_slab = s0;
    U::aim(a, in_unit, w);
    auto ahead = [&]() __attribute__((always_inline)) {
        if (in_unit >= units || s0 == s1) return;
        ring.issue(w, w, 128u * (uint32_t)in_slab, row_bytes - 128 * in_slab);
        if (++in_slab == s1) {
            in_slab = s0;
            in_unit += (int)gridDim.x;
            if (in_unit < units) U::aim(a, in_unit, w);
        }
    };
    SlabFrag<E> x[TB][SLABS];
    const __amdgpu_buffer_rsrc_t xbuf = panel(a.X);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const uint32_t row = (uint32_t)min((int64_t)(16 * t + (lane & 15)), a.M - 1) * (uint32_t)(a.ldx * sizeof(E));
#pragma unroll
        for (int j = 0; j < SLABS; ++j)  // slabs past s1 are not used
            x[t][j] = slab_load<E>(xbuf, row, 128u * (uint32_t)(s0 + j), row_bytes - 128 * (s0 + j));
    }
    // loads return in order: with the tokens first, the first slab is multiplied
    // as soon as it lands
    asm volatile("" ::: "memory");
#pragma unroll 1
    for (int p = 0; p < ring.DEPTH; ++p) ahead();

    int parity = 0, first = 0;
    for (int u = blockIdx.x; u < units; u += (int)gridDim.x) {
        f32x4 acc[TB] = {};
        unroll_seq<SLABS>([&](auto j) __attribute__((always_inline)) {
            if (s0 + (int)j >= s1) return;
            SlabFrag<E> fw, unused;
            ring.take(fw, unused);
            ahead();
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[t] = slab_product(acc[t], fw, x[t][j]);
        });
        if constexpr (TB > 1) __syncthreads();  // one set of sums: the last unit's have been read
#pragma unroll
        for (int t = 0; t < TB; ++t) U::put(sums[parity][t][wave], acc[t]);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TB; ++t) U::finish(a, u, 16 * t, sums[parity][t], (tid - first) & (64 * kWaves - 1));
        first += 16 * U::R;  // the next unit is finished by other wavefronts
        if constexpr (TB == 1) parity ^= 1;  // one set is read while the next unit's is written
    }
}

// Tokens in the ring: any number, any K.
template <typename E, typename O, bool GATED>
__global__ __launch_bounds__(64 * kWaves) void skinny_ring_kernel(LinearArgs<E, O> a, int units, int groups) {
    using U = Unit<E, O, GATED>;
    __shared__ __align__(16) char ring_mem[kWaves * kRingBytes];
    __shared__ __align__(16) float sums[2][kWaves][16 * kSumStride];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row_bytes = (int)(a.K * (int)sizeof(E));
    int s0, s1;
    my_slabs(row_bytes, wave, s0, s1);

    // the stream: slabs s0 .. s1 of segment after segment (unit, token group)
    SlabRows w, x;
    SlabRing<E, true> ring{ring_mem + wave * kRingBytes};
    int in_unit = blockIdx.x, in_group = 0, in_slab = s0;
    auto aim_tokens = [&]() __attribute__((always_inline)) {
        const int64_t t0 = 16 * (int64_t)in_group;
        const int last = (int)min((int64_t)16, a.M - t0) - 1;
        x.buf[0] = x.buf[1] = panel(a.X + t0 * a.ldx);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            x.off[q] = (uint32_t)min(slab_row(q), last) * (uint32_t)(a.ldx * sizeof(E)) + slab_chunk(q);
    };
    U::aim(a, in_unit, w);
    aim_tokens();
    auto ahead = [&]() __attribute__((always_inline)) {
        if (in_unit >= units || s0 == s1) return;
        ring.issue(w, x, 128u * (uint32_t)in_slab, row_bytes - 128 * in_slab);
        if (++in_slab == s1) {
            in_slab = s0;
            if (++in_group == groups) {
                in_group = 0;
                in_unit += (int)gridDim.x;
                if (in_unit < units) U::aim(a, in_unit, w);
            }
            aim_tokens();
        }
    };
#pragma unroll 1
    for (int p = 0; p < ring.DEPTH; ++p) ahead();

    int parity = 0, first = 0;
    for (int u = blockIdx.x; u < units; u += (int)gridDim.x) {
        for (int tg = 0; tg < groups; ++tg, parity ^= 1) {
            f32x4 acc = {};
#pragma unroll 1
            for (int s = s0; s < s1; ++s) {
                SlabFrag<E> fw, fx;
                ring.take(fw, fx);
                ahead();
                acc = slab_product(acc, fw, fx);
            }
            U::put(sums[parity][wave], acc);
            __syncthreads();
            U::finish(a, u, 16 * (int64_t)tg, sums[parity], (tid - first) & (64 * kWaves - 1));
            first += 16 * U::R;
        }
    }
}

// Workgroups: at most one per CU, the same number of units each (224 x 4 units
// rather than 128 x 4 and 128 x 3).
inline unsigned balanced(int units) {
    const int rounds = (units + 255) / 256;
    return (unsigned)((units + rounds - 1) / rounds);
}

template <typename E, typename O, bool GATED, int SLABS, int TB>
hipError_t launch_slabs(const LinearArgs<E, O> &a, int units, hipStream_t st) {
    hipLaunchKernelGGL((skinny_kernel<E, O, GATED, SLABS, TB>), dim3(balanced(units)), dim3(64 * kWaves),
                       0, st, a, units);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_skinny(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    const int units = (int)((a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16));
    const int slabs = (int)((a.K * (int64_t)sizeof(E) + 128 * kWaves - 1) / (128 * kWaves));  // of a wavefront
    // registers hold the tokens up to 24 slabs of 16 tokens or 12 of 32
    if (a.M <= 16 && slabs <= 24) {
        if (slabs <= 2) return launch_slabs<E, O, GATED, 2, 1>(a, units, st);
        if (slabs <= 4) return launch_slabs<E, O, GATED, 4, 1>(a, units, st);
        if (slabs <= 8) return launch_slabs<E, O, GATED, 8, 1>(a, units, st);
        if (slabs <= 16) return launch_slabs<E, O, GATED, 16, 1>(a, units, st);
        return launch_slabs<E, O, GATED, 24, 1>(a, units, st);
    }
    if (a.M <= 32 && slabs <= 12) {
        if (slabs <= 4) return launch_slabs<E, O, GATED, 4, 2>(a, units, st);
        if (slabs <= 8) return launch_slabs<E, O, GATED, 8, 2>(a, units, st);
        return launch_slabs<E, O, GATED, 12, 2>(a, units, st);
    }
    hipLaunchKernelGGL((skinny_ring_kernel<E, O, GATED>), dim3(balanced(units)), dim3(64 * kWaves), 0, st,
                       a, units, (int)((a.M + 15) / 16));
    return hipGetLastError();
}

template hipError_t launch_skinny<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_skinny<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_skinny<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
