// Linear layer and gated pair for few tokens, bound by reading the weights once.
//
// A workgroup takes units of 16 weight rows (16 output features, or 8 gate and
// the same 8 up rows) and streams them through its wavefronts' rings (skinny.h);
// a unit's epilogue runs while the next unit's slabs are landing.  Where it has
// several units, tokens that fit stay in registers (skinny_kernel): 16 and 32 tokens,
// gated 4096 -> 14336 (235 MB of weights), 43 and 47.5 us against 46 and 74.  Others go
// through the ring beside the weights, in groups of 16 on the same unit
// (skinny_ring_kernel): loading 16 or 32 rows into registers takes 2 to 4 us before
// the first product, 16 tokens, 4096 -> 4096 8.0 us against 10.0, 11008 -> 4096 18.2
// against 23.2; 32 tokens, 1024 -> 1024 5.0 against 7.2.
#include "skinny.h"

namespace dyra {

namespace {

// Units of 16 weight rows: where they lie, and what becomes of their sums.
template <typename E, typename O, bool GATED> struct Units {
    static constexpr int R = GATED ? 8 : 16;  // output features
    const LinearArgs<E, O> *a;
    __device__ __forceinline__ void weights(int unit, SlabRows &w, bool fresh) const {
        // rows past the last one lie past the end of the buffer
        const int64_t from = (int64_t)unit * R * a->ldw;
        const int64_t bytes = ((a->N - 1) * a->ldw + a->K - from) * (int64_t)sizeof(E);
        w.buf[0] = panel(a->W0 + from, bytes);
        w.buf[1] = GATED ? panel(a->W1 + from, bytes) : w.buf[0];
        if (!fresh) return;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w.off[q] = (uint32_t)(GATED ? slab_row(q) & 7 : slab_row(q)) * (uint32_t)(a->ldw * sizeof(E)) + slab_chunk();
    }
    // What goes through the ring beside them: tokens 16 group ..
    static constexpr bool kPaired = false;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t other(int group) const {
        const int64_t from = 16 * (int64_t)group * a->ldx;
        return panel(a->X + from, ((a->M - 1) * a->ldx + a->K - from) * (int64_t)sizeof(E));
    }
    __device__ __forceinline__ int64_t other_ld() const { return a->ldx; }
    __device__ __forceinline__ void finish_group(int unit, int group, const float *sums, int thread) const {
        finish(unit, 16 * (int64_t)group, sums, thread, 16);
    }
    static constexpr int kGroupFinishers = 16 * R;
    // Token t and feature f of the unit, from token `first` on.
    __device__ __forceinline__ void finish(int unit, int64_t first, const float *sums, int thread, int tokens) const {
        const int f = thread % R, t = thread / R;
        const int64_t tok = first + t, c = (int64_t)unit * R + f;
        if (t >= tokens || tok >= a->M || c >= a->N) return;
        const float *block = sums + (t >> 4) * kWaves * kBlockSums;
        float y[1] = {joined(block, t & 15, f) + (a->b0 ? to_f32(a->b0[c]) : 0.f)};
        activate<sizeof(O) == 4>(y, a->act);
        if constexpr (GATED) y[0] *= joined(block, t & 15, 8 + f) + (a->b1 ? to_f32(a->b1[c]) : 0.f);
        else if (a->R) y[0] += to_f32(a->R[tok * a->ldr + c]);
        a->Y[tok * a->ldy + c] = to_elem<O>(y[0]);
    }
};

template <typename E, typename O, bool GATED, int TB> struct UnitPosition {
    static constexpr int kFinishers = 16 * TB * Units<E, O, GATED>::R;
    Units<E, O, GATED> units;
    int left, unit;
    __device__ UnitPosition(const LinearArgs<E, O> &a, int n) : units{&a}, unit((int)blockIdx.x) {
        left = (n - unit + (int)gridDim.x - 1) / (int)gridDim.x;
    }
    __device__ __forceinline__ void advance() { unit += (int)gridDim.x; }
    __device__ __forceinline__ void weights(SlabRows &w, bool fresh) const { units.weights(unit, w, fresh); }
    __device__ __forceinline__ bool new_tokens() const { return false; }
    __device__ __forceinline__ int blocks() const { return TB; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t tokens() const { return panel(units.a->X); }
    __device__ __forceinline__ uint32_t token_row(int t) const {
        const int r = 16 * t + (threadIdx.x & 15);
        return r < units.a->M ? (uint32_t)r * (uint32_t)(units.a->ldx * sizeof(E)) : kOutside;
    }
    __device__ __forceinline__ void finish(const float *sums, int thread) const {
        units.finish(unit, 0, sums, thread, 16 * TB);
    }
};

template <typename E, typename O, bool GATED, int SLABS, int TB>
__global__ __launch_bounds__(kThreads) void skinny_kernel(LinearArgs<E, O> a, int units) {
    __shared__ __align__(16) StreamLds<TB> lds;
    const UnitPosition<E, O, GATED, TB> start(a, units);
    stream_products<E, SLABS, TB>(start, (int)(a.K * (int)sizeof(E)), lds);
}

template <typename E, typename O, class U_>
__global__ __launch_bounds__(kThreads) void skinny_ring_kernel(LinearArgs<E, O> a, int units, int groups) {
    __shared__ __align__(16) StreamLds<1> lds;
    const U_ U{&a};
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row_bytes = (int)(a.K * (int)sizeof(E));
    const int slabs = (row_bytes + 127) / 128, per = (slabs + kWaves - 1) / kWaves;
    const int s0 = min(slabs, wave * per), s1 = min(slabs, s0 + per);  // this wavefront's slabs

    // the stream: slabs s0 .. s1 of segment after segment (unit, token group)
    SlabRing<E, 16, 16> ring{lds.ring + wave * kRingBytes};
    SlabRows w, x;
    const uint32_t xld = (uint32_t)(U.other_ld() * sizeof(E));
#pragma unroll
    for (int q = 0; q < 2; ++q) x.off[q] = (uint32_t)slab_row(q) * xld + slab_chunk();
    int in_unit = s0 < s1 ? (int)blockIdx.x : units, in_group = 0, in_slab = s0;
    auto aim_tokens = [&]() __attribute__((always_inline)) { x.buf[0] = x.buf[1] = U.other(in_group); };
    U.weights(min(in_unit, units - 1), w, true);
    aim_tokens();
    auto ahead = [&]() __attribute__((always_inline)) {
        ring.issue(w, x, 128u * (uint32_t)in_slab, in_unit < units ? row_bytes - 128 * in_slab : 0);
        if (++in_slab >= s1) {
            in_slab = s0;
            if (++in_group == groups) {
                in_group = 0;
                in_unit += (int)gridDim.x;
                if (in_unit < units) U.weights(in_unit, w, false);
            }
            if (groups > 1) aim_tokens();
        }
    };
#pragma unroll 1
    for (int q = 0; q < ring.DEPTH; ++q) ahead();

    int set = 0, begin = 0;
    for (int u = blockIdx.x; u < units; u += (int)gridDim.x) {
        for (int group = 0; group < groups; ++group, set ^= 1) {
            f32x4 acc = {};
#pragma unroll 1
            for (int s = s0; s < s1; ++s) {
                SlabFrag<E> fw, fx;
                ring.take(fw, fx);
                ahead();
                acc = slab_product(acc, fw, fx);
            }
            // two sets of sums: one is read while the next segment's is written; paired,
            // both are read at the end of the second
            if (U.kPaired && group == 0) __syncthreads();
            *reinterpret_cast<f32x4 *>(&lds.sums[set][wave][(lane & 15) * 16 + 4 * (lane >> 4)]) = acc;
            __syncthreads();
            if (U.kPaired && group == 0) continue;
            U.finish_group(u, group, &lds.sums[U.kPaired ? 0 : set][0][0], (tid - begin) & (kThreads - 1));
            begin += U.kGroupFinishers;  // other wavefronts finish the next one
        }
    }
    wait_vmcnt<0>();
}

// Few features (32, gated 16 pairs) of many tokens, as of a router or a small head:
// the same ring with the operands' roles exchanged: a unit is 16 rows of X, the
// groups are the weights' rows 0 .. 15 and 16 .. 31, or gate and up.  Tiles, which
// do not split K, would fill few CUs.
template <typename E, typename O, bool GATED> struct NarrowUnits {
    const LinearArgs<E, O> *a;
    __device__ __forceinline__ void weights(int unit, SlabRows &w, bool fresh) const {
        const int64_t from = 16 * (int64_t)unit * a->ldx;
        w.buf[0] = w.buf[1] = panel(a->X + from, ((a->M - 1) * a->ldx + a->K - from) * (int64_t)sizeof(E));
        if (!fresh) return;
#pragma unroll
        for (int q = 0; q < 2; ++q) w.off[q] = (uint32_t)slab_row(q) * (uint32_t)(a->ldx * sizeof(E)) + slab_chunk();
    }
    static constexpr bool kPaired = GATED;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t other(int group) const {
        const int64_t from = GATED ? 0 : 16 * (int64_t)group * a->ldw;
        return panel((GATED && group == 1 ? a->W1 : a->W0) + from,
                     ((a->N - 1) * a->ldw + a->K - from) * (int64_t)sizeof(E));
    }
    __device__ __forceinline__ int64_t other_ld() const { return a->ldw; }
    static constexpr int kGroupFinishers = 256;
    // Features 16 group .. (gated: all, from the sums of gate and up) of the unit's tokens.
    __device__ __forceinline__ void finish_group(int unit, int group, const float *sums, int thread) const {
        const int f = thread & 15, i = thread >> 4;
        const int64_t tok = 16 * (int64_t)unit + i, c = (GATED ? 0 : 16 * group) + f;
        if (i >= 16 || tok >= a->M || c >= a->N) return;
        float y[1] = {joined(sums, f, i) + (a->b0 ? to_f32(a->b0[c]) : 0.f)};
        activate<sizeof(O) == 4>(y, a->act);
        if constexpr (GATED) y[0] *= joined(sums + kWaves * kBlockSums, f, i) + (a->b1 ? to_f32(a->b1[c]) : 0.f);
        else if (a->R) y[0] += to_f32(a->R[tok * a->ldr + c]);
        a->Y[tok * a->ldy + c] = to_elem<O>(y[0]);
    }
};

// At most one workgroup per CU, the same number of units each (224 x 4 units
// rather than 128 x 4 and 128 x 3: 16 tokens, 4096 -> 14336, 29.4 -> 24.4 us).
inline unsigned workgroups(int units) {
    const int rounds = (units + 255) / 256;
    return (unsigned)((units + rounds - 1) / rounds);
}

template <typename E, typename O, bool GATED, int SLABS, int TB>
hipError_t launch_slabs(const LinearArgs<E, O> &a, int units, hipStream_t st) {
    hipLaunchKernelGGL((skinny_kernel<E, O, GATED, SLABS, TB>), dim3(workgroups(units)), dim3(kThreads), 0, st, a, units);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_skinny(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    const int units = (int)few_token_units(GATED, a.N);
    const FewTokens few = few_tokens(GATED, a.M, a.N, a.K * (int64_t)sizeof(E));
    static_assert(kWaves == 8, "few_tokens divides K by it");
    if (few.blocks == 1) {
        switch (few.slabs) {
        case 2: return launch_slabs<E, O, GATED, 2, 1>(a, units, st);
        case 4: return launch_slabs<E, O, GATED, 4, 1>(a, units, st);
        case 8: return launch_slabs<E, O, GATED, 8, 1>(a, units, st);
        case 16: return launch_slabs<E, O, GATED, 16, 1>(a, units, st);
        case 24: return launch_slabs<E, O, GATED, 24, 1>(a, units, st);
        }
    } else {
        switch (few.slabs) {
        case 4: return launch_slabs<E, O, GATED, 4, 2>(a, units, st);
        case 8: return launch_slabs<E, O, GATED, 8, 2>(a, units, st);
        case 12: return launch_slabs<E, O, GATED, 12, 2>(a, units, st);
        }
    }
    hipLaunchKernelGGL((skinny_ring_kernel<E, O, Units<E, O, GATED>>), dim3(workgroups(units)), dim3(kThreads), 0, st, a,
                       units, (int)((a.M + 15) / 16));
    return hipGetLastError();
}

template <typename E, typename O, bool GATED> hipError_t launch_narrow(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    const int units = (int)((a.M + 15) / 16);
    hipLaunchKernelGGL((skinny_ring_kernel<E, O, NarrowUnits<E, O, GATED>>), dim3(workgroups(units)), dim3(kThreads), 0,
                       st, a, units, GATED || a.N > 16 ? 2 : 1);
    return hipGetLastError();
}

template hipError_t launch_skinny<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_narrow<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_narrow<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_skinny<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_narrow<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_skinny<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_narrow<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<float, float, true>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_narrow<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
