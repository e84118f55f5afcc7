// Rows on their way to a product in 8-bit integers: the root-mean-square norm with
// the residual's addition, quantisation, and back.
//
//     z = x + r,  rho = 1 / sqrt(mean z^2 + eps),  y = z rho w
//     a = max |y| = rho max |z w|,  s = max(a, 127 2^-126) / 127,  q = nearest(y / s)
//
// The sum of squares and max |z w| do not wait for one another, so a row needs one
// reduction.  s is taken from a normal float32 at least (2^-126 for a row of zeros).  q is
// 127 y / a (Steps), of which rho is no part: z w is measured by its own largest.  A row
// whose a is not finite has s = NaN and q = 0: what is made of it is NaN.
//
// Squares past float32's range (|z| > 1.8e19) are summed again with z 2^-96, whose norm is
// the same up to eps 2^-192, which is nothing beside them.  Results are made of z 2^-48, so
// that small values of such a row keep their bits.
#include "ffn_tile.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace dyra {

namespace {

constexpr float kLeastTop = 127.f * FLT_MIN;
// Threads of a launch along its first dimension: below 2^32.  More rows take more launches.
constexpr int64_t kLaunchThreads = int64_t{1} << 31;

// What a row's threads find together: the sum of squares, and the largest magnitude as
// its bits, which order as the magnitudes do with NaN above infinity.
struct RowStats {
    float sum;
    unsigned top;
};
// Joined over the THREADS of a row: neighbouring lanes of one wavefront, or a workgroup's
// wavefronts, which all call it.
template <int THREADS> __device__ __forceinline__ RowStats joined_row(RowStats v) {
#pragma unroll
    for (int d = (THREADS < 64 ? THREADS : 64) / 2; d > 0; d >>= 1) {
        v.sum += __shfl_xor(v.sum, d);
        v.top = max(v.top, (unsigned)__shfl_xor((int)v.top, d));
    }
    if constexpr (THREADS > 64) {
        constexpr int W = THREADS / 64;
        __shared__ float sums[W];
        __shared__ unsigned tops[W];
        __syncthreads();  // the last ones have been read
        if ((threadIdx.x & 63) == 0) {
            sums[threadIdx.x >> 6] = v.sum;
            tops[threadIdx.x >> 6] = v.top;
        }
        __syncthreads();
        v = {0.f, 0u};
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v.sum += sums[i];
            v.top = max(v.top, tops[i]);
        }
    }
    return v;
}

// V elements as they lie in memory (16 bytes), any alignment of their type.  Results are
// stored non-temporally: they do not push out of the L2 what other workgroups are about to
// read (16384 x 4096 bf16, norm with residual to 8 bits 81.5 us without, 76.2 with, to bf16 91
// and 85, dequantisation 33.7 and 29.5).  Loads of that kind gain less and cost a few us where X
// still lies in a cache.
template <typename E> struct Chunk {
    static constexpr int V = 16 / (int)sizeof(E);
    union {
        u32x4 u;
        E e[V];
    };
    __device__ __forceinline__ void load(const E *p) { u = *reinterpret_cast<const u32x4_any *>(p); }
    __device__ __forceinline__ void store(E *p) const { __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any *>(p)); }
};

// 127 y / top to the nearest whole number, halves to the even one, in a float32's low bits.
// In bf16 rows every value of half the largest is such a half, so the ratio has to be right to
// better than a float32 rounding: y steps alone is off by up to 2^-24 of itself, and those
// values went to 63 or 64 as 127 / top happened to be rounded.  `rest`, what that rounding
// left out, puts the ratio right to 2^-46 before its one rounding, and still to 2^-28 where
// rest is subnormal (top above 2^102).  Two operations more a value, under the loads of long
// rows: us without | with, bf16: 16384 x 14336 123.5 | 123.5, 2048 x 65536 (a row a CU) 75.2 |
// 76.1, 16 x 14336 3.4 | 3.5, norms of 32768 x 200 7.4 | 7.8.
struct Steps {
    float steps, rest;
    // top: 127 2^-126 .. 2^128, so that 127 / top is a normal float32 too
    __device__ __forceinline__ explicit Steps(float top) : steps(127.f / top) {
        rest = __builtin_fmaf(-steps, top, 127.f) * (1.f / 127.f) * steps;
    }
    __device__ __forceinline__ unsigned of(float y) const {
        const float ratio = __builtin_fmaf(y, steps, y * rest);
        return __float_as_uint(ratio + 12582912.f);  // 1.5 2^23: its last place is 1
    }
};
// The low bytes of four.
__device__ __forceinline__ unsigned bytes4(unsigned a, unsigned b, unsigned c, unsigned d) {
    const unsigned lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
    return lo | hi << 16;
}
// Of V values, with `keep` 0 as zeros.
template <int V> __device__ __forceinline__ void store_bytes(i8 *p, const unsigned (&q)[V], unsigned keep) {
    typedef unsigned u32_any __attribute__((aligned(1)));
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    typedef u32x2 u32x2_any __attribute__((aligned(1)));
    const unsigned lo = bytes4(q[0], q[1], q[2], q[3]) & keep;
    if constexpr (V == 4) __builtin_nontemporal_store(lo, reinterpret_cast<u32_any *>(p));
    else __builtin_nontemporal_store(u32x2{lo, bytes4(q[4], q[5], q[6], q[7]) & keep}, reinterpret_cast<u32x2_any *>(p));
}

// Threads of a workgroup: rows within a wavefront share one, longer rows have their own.
constexpr int rows_threads(int row) { return row <= 64 ? 256 : row; }

// THREADS threads hold a row of up to THREADS * CHUNKS whole 16-byte chunks, and one
// more element each of the rest: it is read once, all its loads in flight together.  Bound
// by memory: 16384 x 4096 bf16 with residual 80 us to 8 bits (5.9 TB/s of read and
// written bytes) and 93 to bf16 (5.8); quantisation 36 us (5.6), 16384 x 14336 124 (5.7).
// One workgroup a row that was read twice, by elements: 255 to 8 bits, 330 the last.
template <typename E, bool NORM, bool EIGHT, int THREADS, int CHUNKS>
__global__ __launch_bounds__(rows_threads(THREADS)) void rows_kernel(RowArgs<E> a) {
    constexpr int V = Chunk<E>::V, ROWS = rows_threads(THREADS) / THREADS;
    int t = threadIdx.x % THREADS;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
    if (ROWS > 1 && row >= a.N) return;  // all threads of a row, which wait for no others
    const int c = (int)a.c, chunks = c / V, rest = chunks * V + t;
    const bool last = rest < c;
    const E *const x = a.X + row * a.ldx, *const r = NORM && a.R ? a.R + row * a.ldr : nullptr;

    // In the longest float32 rows z alone is 64 of a thread's 128 registers.  X and the residual are
    // loaded half of the chunks at a time, weights four chunks at a time, and a chunk's place is
    // computed anew for each use: without that 32 to 47 registers went to scratch.  us without |
    // with, 2048 x 65536: norm 300 | 209, with residual 484 | 404 (5.3 TB/s), to 8 bits 320 | 183,
    // with residual 485 | 363 (4.8 TB/s).
    constexpr bool TIGHT = NORM && CHUNKS > 8;
    constexpr int AT_ONCE = TIGHT ? CHUNKS / 2 : CHUNKS;
    auto fresh = [&]() __attribute__((always_inline)) {
        if (TIGHT) {
            asm volatile("" : "+v"(t));
            t &= THREADS - 1;
        }
    };
    float z[CHUNKS][V], z1 = 0.f;
    if (last) z1 = to_f32(x[rest]) + (r ? to_f32(r[rest]) : 0.f);
#pragma unroll
    for (int from = 0; from < CHUNKS; from += AT_ONCE) {
        Chunk<E> xs[AT_ONCE], rs[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            xs[i].u = rs[i].u = u32x4{};
            const int k = t + (from + i) * THREADS;
            if (k < chunks) {
                xs[i].load(x + k * V);
                if (r) rs[i].load(r + k * V);
            }
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                z[from + i][q] = to_f32(xs[i].e[q]) + (r ? to_f32(rs[i].e[q]) : 0.f);
                if (TIGHT) asm volatile("" : "+v"(z[from + i][q]));  // made here, before the other half is asked for
            }
        fresh();
    }
    if (NORM && a.S) {
        E *const s = a.S + row * a.lds;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int k = t + i * THREADS;
            if (k < chunks) {
                Chunk<E> o;
#pragma unroll
                for (int q = 0; q < V; ++q) o.e[q] = to_elem<E>(z[i][q]);
                o.store(s + k * V);
            }
        }
        if (last) s[rest] = to_elem<E>(z1);
    }

    // The longest rows' weights are read again where they are used, the others held.
    constexpr bool HELD = CHUNKS * V * THREADS < 65536;
    Chunk<E> ws[HELD ? CHUNKS : 1];
    float w1 = 1.f;
    const bool weighted = NORM && a.W;
    auto load_weights = [&](int i) __attribute__((always_inline)) {
        Chunk<E> &w = ws[HELD ? i : 0];
        w.u = u32x4{};
        const int k = t + i * THREADS;
        if (k < chunks) w.load(a.W + k * V);
    };
    if (weighted) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) load_weights(i);
        }
        if (last) w1 = to_f32(a.W[rest]);
    }
    // before the first use of a chunk's weights
    auto weights = [&](int i) __attribute__((always_inline)) {
        if (!HELD && weighted) {
            asm volatile("" ::: "memory");
            load_weights(i);
        }
    };
    auto weight = [&](int i, int q) { return weighted ? to_f32(ws[HELD ? i : 0].e[q]) : 1.f; };
    auto stats = [&](float by) {
        RowStats v = {0.f, 0u};
        fresh();
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            if (EIGHT) weights(i);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float y = z[i][q] * by;
                if (NORM) v.sum = __builtin_fmaf(y, y, v.sum);
                if (EIGHT) v.top = max(v.top, __float_as_uint(y * weight(i, q)) & 0x7fffffffu);
            }
            if (TIGHT && i % 4 == 3) asm volatile("" : "+v"(v.top));  // four chunks of weights at a time
        }
        if (NORM) v.sum = __builtin_fmaf(z1 * by, z1 * by, v.sum);
        if (EIGHT) v.top = max(v.top, __float_as_uint(z1 * by * w1) & 0x7fffffffu);
        return joined_row<THREADS>(v);
    };
    float by = 1.f, rho = 1.f;
    RowStats v = stats(1.f);
    if constexpr (NORM) {
        if (!(v.sum < INFINITY)) {
            by = 0x1p-96f;
            v = stats(by);
        }
        rho = 1.f / sqrtf(v.sum / (float)c + a.eps * (by * by));
    }
    if constexpr (EIGHT) {
        // Where z w leaves float32's range or nears its end, or the scale its least value, y is measured
        // itself, (z rho) w: rows of zeros and of infinities too.
        const float zw = __uint_as_float(v.top);
        if (NORM && !(zw * rho >= kLeastTop && zw >= 0x1p-100f && zw < INFINITY)) {
            by *= rho;
            rho = 1.f;
            v = stats(by);
        }
        const float most = __uint_as_float(v.top), largest = most * rho;
        const bool finite = v.top < 0x7f800000u && largest < INFINITY;
        if (t == 0) a.scales[row] = finite ? fmaxf(largest, kLeastTop) / 127.f : NAN;
        const Steps to(fmaxf(most, kLeastTop));
        fresh();
        const unsigned keep = finite ? 0xffffffffu : 0u;
        i8 *const y = (i8 *)a.Y + row * a.ldy;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int k = t + i * THREADS;
            weights(i);
            if (k < chunks) {
                unsigned b[V];
#pragma unroll
                for (int q = 0; q < V; ++q) b[q] = to.of(z[i][q] * by * weight(i, q));
                store_bytes<V>(y + k * V, b, keep);
            }
        }
        if (last) y[rest] = (i8)(to.of(z1 * by * w1) & keep);
    } else {
        if (by < 1.f) {  // the other half of 2^-96 goes into rho: z by is subnormal only where z rho is
            by = 0x1p-48f;
            rho *= by;
        }
        fresh();
        E *const y = (E *)a.Y + row * a.ldy;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int k = t + i * THREADS;
            weights(i);
            if (k < chunks) {
                Chunk<E> o;
#pragma unroll
                for (int q = 0; q < V; ++q) o.e[q] = to_elem<E>(z[i][q] * by * rho * weight(i, q));
                o.store(y + k * V);
            }
        }
        if (last) y[rest] = to_elem<E>(z1 * by * rho * w1);
    }
}

// Back: 16 bytes of results a thread, THREADS threads to a piece of a row.
template <typename E, int THREADS>
__global__ __launch_bounds__(256) void dequantize_kernel(const i8 *Q, int64_t ldq, const float *scales, int64_t N, int c, E *X,
                                                         int64_t ldx) {
    constexpr int V = Chunk<E>::V, ROWS = 256 / THREADS;
    typedef unsigned u32xn __attribute__((ext_vector_type(V / 4)));
    typedef u32xn u32xn_any __attribute__((aligned(1)));
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
    if (row >= N) return;
    const int at = V * ((int)threadIdx.x % THREADS + (int)blockIdx.y * THREADS);
    const i8 *const from = Q + row * ldq;
    E *const to = X + row * ldx;
    const float s = scales[row];
    if (at + V <= c) {
        union {
            u32xn u;
            i8 e[V];
        } q;
        q.u = *reinterpret_cast<const u32xn_any *>(from + at);
        Chunk<E> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.e[j] = to_elem<E>((float)q.e[j] * s);
        o.store(to + at);
    } else {
        for (int j = at; j < c; ++j) to[j] = to_elem<E>((float)from[j] * s);
    }
}

template <typename E, bool NORM, bool EIGHT, int THREADS, int CHUNKS>
hipError_t launch_held(RowArgs<E> a, hipStream_t st) {
    constexpr int ROWS = rows_threads(THREADS) / THREADS;
    constexpr int64_t MOST = kLaunchThreads / THREADS;  // rows of a launch
    typedef std::conditional_t<EIGHT, i8, E> Out;
    for (int64_t left = a.N; left > 0; left -= MOST) {
        a.N = std::min(left, MOST);
        hipLaunchKernelGGL((rows_kernel<E, NORM, EIGHT, THREADS, CHUNKS>), dim3((unsigned)((a.N + ROWS - 1) / ROWS)),
                           dim3(rows_threads(THREADS)), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= MOST) return e;
        a.X += MOST * a.ldx;
        if (a.R) a.R += MOST * a.ldr;
        if (a.S) a.S += MOST * a.lds;
        a.Y = (Out *)a.Y + MOST * a.ldy;
        if (EIGHT) a.scales += MOST;
    }
    return hipSuccess;
}
// Two chunks a thread while that gives threads enough: more loads in flight than with one,
// more threads than with four.  us by threads x chunks of a row, norm with residual to 8
// bits, bf16: 16384 x 4096 256 x 2 81.5, 128 x 4 83.4, 512 x 1 83.6, 64 x 8 92.3; 25728 x
// 1024 64 x 2 36.4, 256 x 1 47.1; 32768 x 64 8 x 1 5.6, 64 x 1 14.7; 20000 x 512 32 x 2
// 14.7, 64 x 1 16.0, 128 x 1 19.1; 8192 x 11008 512 x 4 114.8, 256 x 8 114.9, 1024 x 2 141.6;
// few rows take 3.6 to 5 us with all of them.
template <typename E, bool NORM, bool EIGHT> hipError_t launch_rows(const RowArgs<E> &a, hipStream_t st) {
    if (a.N <= 0) return hipSuccess;
    constexpr int V = Chunk<E>::V;
    const int64_t chunks = a.c / V;
    if (chunks <= 8) return launch_held<E, NORM, EIGHT, 8, 1>(a, st);
    if (chunks <= 32) return launch_held<E, NORM, EIGHT, 16, 2>(a, st);
    if (chunks <= 64) return launch_held<E, NORM, EIGHT, 32, 2>(a, st);
    if (chunks <= 128) return launch_held<E, NORM, EIGHT, 64, 2>(a, st);
    if (chunks <= 256) return launch_held<E, NORM, EIGHT, 128, 2>(a, st);
    if (chunks <= 512) return launch_held<E, NORM, EIGHT, 256, 2>(a, st);
    if (chunks <= 1024) return launch_held<E, NORM, EIGHT, 512, 2>(a, st);
    if (chunks <= 2048) return launch_held<E, NORM, EIGHT, 512, 4>(a, st);
    if (chunks <= 4096) return launch_held<E, NORM, EIGHT, 1024, 4>(a, st);
    if (chunks <= 8192) return launch_held<E, NORM, EIGHT, 1024, 8>(a, st);
    if constexpr (V == 4) return launch_held<E, NORM, EIGHT, 1024, 16>(a, st);
    return hipErrorInvalidValue;  // longer rows are refused
}

template <typename E, int THREADS>
hipError_t launch_back(const i8 *Q, int64_t ldq, const float *scales, int64_t N, int64_t c, E *X, int64_t ldx, hipStream_t st) {
    constexpr int ROWS = 256 / THREADS, PIECE = Chunk<E>::V * THREADS;
    constexpr int64_t MOST = kLaunchThreads / THREADS;
    for (int64_t from = 0; from < N; from += MOST) {
        const int64_t rows = std::min(N - from, MOST);
        hipLaunchKernelGGL((dequantize_kernel<E, THREADS>),
                           dim3((unsigned)((rows + ROWS - 1) / ROWS), (unsigned)((c + PIECE - 1) / PIECE)), dim3(256), 0, st,
                           Q + from * ldq, ldq, scales + from, rows, (int)c, X + from * ldx, ldx);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
    // us by threads of a piece, bf16: 25728 x 200 16 4.9, 64 6.0, 256 9.5; 25728 x 1024 64
    // 15.5, 256 18.6; 16384 x 4096 256 33.6, 64 41.2
    constexpr int V = Chunk<E>::V;
    if (c <= 16 * V) return launch_back<E, 16>(Q, ldq, scales, N, c, X, ldx, st);
    if (c <= 32 * V) return launch_back<E, 32>(Q, ldq, scales, N, c, X, ldx, st);
    if (c <= 128 * V) return launch_back<E, 64>(Q, ldq, scales, N, c, X, ldx, st);
    return launch_back<E, 256>(Q, ldq, scales, N, c, X, ldx, st);
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
