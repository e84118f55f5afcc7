// Rows on their way to a product in 8-bit integers: the root-mean-square norm with
// the residual's addition, quantisation, and back.
//
//     z = x + r,  rho = 1 / sqrt(mean z^2 + eps),  y = z rho w
//     a = max |y| = rho max |z w|,  s = max(a, 127 2^-126) / 127,  q = nearest(y / s)
//
// The sum of squares and max |z w| do not wait for one another, so a row needs one
// reduction.  s is taken from a normal float32 at least (2^-126 for a row of zeros): y / s
// is y (127 / a), and neither factor leaves float32's range.  A row whose a is not finite
// has s = NaN and q = 0: what is made of it is NaN.
//
// Squares past float32's range (|z| > 1.8e19) are summed again with z 2^-96, whose norm is
// the same up to eps 2^-192, which is nothing beside them.
#include "ffn_tile.h"

#include <cfloat>
#include <cmath>

namespace dyra {

namespace {

constexpr int kRowThreads = 256;
constexpr float kLeastTop = 127.f * FLT_MIN;

// What a row's threads find together: the sum of squares, and the largest magnitude as
// its bits, which order as the magnitudes do with NaN above infinity.
struct RowStats {
    float sum;
    unsigned top;
};
__device__ __forceinline__ RowStats joined_row(RowStats v) {
    __shared__ float sums[kRowThreads / 64];
    __shared__ unsigned tops[kRowThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        v.sum += __shfl_xor(v.sum, d);
        v.top = max(v.top, (unsigned)__shfl_xor((int)v.top, d));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        sums[threadIdx.x >> 6] = v.sum;
        tops[threadIdx.x >> 6] = v.top;
    }
    __syncthreads();
    v = {0.f, 0u};
#pragma unroll
    for (int i = 0; i < kRowThreads / 64; ++i) {
        v.sum += sums[i];
        v.top = max(v.top, tops[i]);
    }
    return v;
}

// One workgroup a row, which is read twice.
template <typename E, bool NORM, bool EIGHT> __global__ __launch_bounds__(kRowThreads) void rows_kernel(RowArgs<E> a) {
    const int64_t row = blockIdx.x;
    const E *x = a.X + row * a.ldx, *r = a.R ? a.R + row * a.ldr : nullptr;
    auto value = [&](int64_t j) { return to_f32(x[j]) + (r ? to_f32(r[j]) : 0.f); };
    auto weight = [&](int64_t j) { return a.W ? to_f32(a.W[j]) : 1.f; };
    auto stats = [&](float by) {
        RowStats v = {0.f, 0u};
        for (int64_t j = threadIdx.x; j < a.c; j += kRowThreads) {
            const float z = value(j) * by;
            v.sum += z * z;
            v.top = max(v.top, __float_as_uint(z * weight(j)) & 0x7fffffffu);
        }
        return joined_row(v);
    };
    float by = 1.f, rho = 1.f;
    RowStats v = stats(by);
    if constexpr (NORM) {
        if (!(v.sum < INFINITY)) {
            by = 0x1p-96f;
            v = stats(by);
        }
        rho = 1.f / sqrtf(v.sum / (float)a.c + a.eps * (by * by));
    }
    const float top = fmaxf(__uint_as_float(v.top) * rho, kLeastTop);
    const bool finite = v.top < 0x7f800000u && top < INFINITY;
    if (EIGHT && threadIdx.x == 0) a.scales[row] = finite ? top / 127.f : NAN;
    const float steps = 127.f / top;
    for (int64_t j = threadIdx.x; j < a.c; j += kRowThreads) {
        const float z = value(j);
        if (NORM && a.S) a.S[row * a.lds + j] = to_elem<E>(z);
        if constexpr (EIGHT) {
            const float y = z * by * weight(j) * rho;
            ((i8 *)a.Y)[row * a.ldy + j] = finite ? (i8)(int)rintf(y * steps) : 0;
        } else {
            ((E *)a.Y)[row * a.ldy + j] = to_elem<E>(z * by * rho * weight(j));
        }
    }
}

template <typename E>
__global__ __launch_bounds__(kRowThreads) void dequantize_kernel(const i8 *Q, int64_t ldq, const float *scales, int64_t c,
                                                                E *X, int64_t ldx) {
    const int64_t row = blockIdx.x;
    const float s = scales[row];
    for (int64_t j = threadIdx.x; j < c; j += kRowThreads) X[row * ldx + j] = to_elem<E>((float)Q[row * ldq + j] * s);
}

template <typename E, bool NORM, bool EIGHT> hipError_t launch_rows(const RowArgs<E> &a, hipStream_t st) {
    if (a.N <= 0) return hipSuccess;
    hipLaunchKernelGGL((rows_kernel<E, NORM, EIGHT>), dim3((unsigned)a.N), dim3(kRowThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

template <typename E> hipError_t launch_norm(const RowArgs<E> &a, hipStream_t st) { return launch_rows<E, true, false>(a, st); }
template <typename E> hipError_t launch_norm_quantize(const RowArgs<E> &a, hipStream_t st) {
    return launch_rows<E, true, true>(a, st);
}
template <typename E> hipError_t launch_quantize(const RowArgs<E> &a, hipStream_t st) { return launch_rows<E, false, true>(a, st); }
template <typename E>
hipError_t launch_dequantize(const i8 *Q, int64_t ldq, const float *scales, int64_t N, int64_t c, E *X, int64_t ldx,
                             hipStream_t st) {
    if (N <= 0) return hipSuccess;
    hipLaunchKernelGGL((dequantize_kernel<E>), dim3((unsigned)N), dim3(kRowThreads), 0, st, Q, ldq, scales, c, X, ldx);
    return hipGetLastError();
}

template hipError_t launch_norm<bf16>(const RowArgs<bf16> &, hipStream_t);
template hipError_t launch_norm<float>(const RowArgs<float> &, hipStream_t);
template hipError_t launch_norm_quantize<bf16>(const RowArgs<bf16> &, hipStream_t);
template hipError_t launch_norm_quantize<float>(const RowArgs<float> &, hipStream_t);
template hipError_t launch_quantize<bf16>(const RowArgs<bf16> &, hipStream_t);
template hipError_t launch_quantize<float>(const RowArgs<float> &, hipStream_t);
template hipError_t launch_dequantize<bf16>(const i8 *, int64_t, const float *, int64_t, int64_t, bf16 *, int64_t, hipStream_t);
template hipError_t launch_dequantize<float>(const i8 *, int64_t, const float *, int64_t, int64_t, float *, int64_t, hipStream_t);

}  // namespace dyra
