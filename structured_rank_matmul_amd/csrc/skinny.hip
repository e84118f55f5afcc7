// Linear layer and gated pair for few tokens, bound by reading the weights
// once.  A workgroup owns 16 output features (of both products when gated) and
// up to 64 tokens; its wavefronts split K, their partial sums meet in LDS in a
// fixed order, and the epilogue runs on the sums.
#include "skinny.h"

#include <algorithm>

namespace dyra {

namespace {

constexpr int kWaves = 8;

template <typename E, typename O, int TN, bool GATED>
__global__ __launch_bounds__(64 * kWaves) void skinny_kernel(LinearArgs<E, O> a) {
    constexpr int MATS = GATED ? 2 : 1;
    __shared__ float red[kWaves][MATS * TN][64][4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int64_t f0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * 16 * TN;
    const int64_t fr = f0 + i16 < a.N ? f0 + i16 : a.N - 1;
    const E *w[MATS], *x[TN];
    w[0] = a.W0 + fr * a.ldw + 8 * g;
    if constexpr (GATED) w[1] = a.W1 + fr * a.ldw + 8 * g;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const int64_t r = t0 + 16 * t + i16;
        x[t] = a.X + (r < a.M ? r : a.M - 1) * a.ldx + 8 * g;
    }
    f32x4 acc[MATS][TN] = {};
    const int steps = (int)((a.K + 31) / 32);
    const int per = (steps + kWaves - 1) / kWaves;
    const int s0 = std::min(steps, wave * per), s1 = std::min(steps, s0 + per);
    skinny_product<E, MATS, TN, 4>(w, x, a.K, s0, s1, acc);
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int t = 0; t < TN; ++t) *reinterpret_cast<f32x4 *>(red[wave][m * TN + t][lane]) = acc[m][t];
    __syncthreads();
    // thread -> (token block, lane of the block): 4 consecutive features of a token
    for (int u = tid; u < 64 * TN; u += 64 * kWaves) {
        const int t = u / 64, l = u % 64;
        const int64_t tok = t0 + 16 * t + (l & 15), c = f0 + 4 * (l >> 4);
        const int have = (int)std::min<int64_t>(4, a.N - c);
        if (tok >= a.M || have <= 0) continue;
        f32x4 z[MATS] = {};
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int v = 0; v < kWaves; ++v) z[m] += *reinterpret_cast<const f32x4 *>(red[v][m * TN + t][l]);
        float y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = z[0][q] + (a.b0 && q < have ? to_f32(a.b0[c + q]) : 0.f);
        activate<sizeof(O) == 4>(y, a.act);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q >= have) continue;
            if constexpr (GATED) y[q] *= z[1][q] + (a.b1 ? to_f32(a.b1[c + q]) : 0.f);
            else if (a.R) y[q] += to_f32(a.R[tok * a.ldr + c + q]);
            a.Y[tok * a.ldy + c + q] = to_elem<O>(y[q]);
        }
    }
}

template <typename E, typename O, int TN, bool GATED> hipError_t launch_tn(const LinearArgs<E, O> &a, hipStream_t st) {
    const int64_t gx = (a.N + 15) / 16, gy = (a.M + 16 * TN - 1) / (16 * TN);
    if (gx > INT32_MAX || gy > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((skinny_kernel<E, O, TN, GATED>), dim3((unsigned)gx, (unsigned)gy), dim3(64 * kWaves), 0, st, a);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_skinny(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    if (a.M <= 16) return launch_tn<E, O, 1, GATED>(a, st);
    if (a.M <= 32) return launch_tn<E, O, 2, GATED>(a, st);
    return launch_tn<E, O, 4, GATED>(a, st);
}

template hipError_t launch_skinny<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_skinny<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_skinny<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
