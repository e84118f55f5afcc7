// Router and expert layer for a few tokens.
//
// Router: a wavefront per row of logits, its values in registers; k rounds of
// an argmax over keys that order by (value, lower index first).
//
// Expert layer, two kernels.  moe_up forms H[pair][f] = act(X Wg_e^T) * (X Wu_e^T)
// for every (token, place) pair; moe_down forms Y = R + sum_j w_j H_j Wd_e^T.
// Both are bound by reading the weights of the chosen experts once: a workgroup
// gathers the tokens of an expert and multiplies them together.  No atomics on
// results: every pair's products have a place of their own in LDS and are added
// per token in the order of its places.
#include "skinny.h"

#include <algorithm>

namespace dyra {

namespace {

// ------------------------------------------------------------------ router

// Orders like the float (-0 as +0), above 0 for every value that may be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename E, int PER>  // PER values per lane: E_n <= 64 PER
__global__ __launch_bounds__(256) void route_kernel(const E *__restrict__ logits, int64_t ld, int64_t T, int En, int k,
                                                    bool sigmoid, bool renormalise, float scale,
                                                    int32_t *__restrict__ ids, float *__restrict__ w) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const E *row = logits + t * ld;
    float v[PER];
    bool ok[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int e = 64 * q + lane;
        v[q] = e < En ? to_f32(row[e]) : -INFINITY;
        ok[q] = v[q] > -INFINITY;  // false for NaN too
    }
    unsigned taken = 0;
    float mine = 0.f;  // lane j: the j-th chosen value and expert
    int my_id = -1;
    float top = 0.f;
    for (int j = 0; j < k; ++j) {
        uint32_t key = 0;
        int at = En;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const uint32_t o = ok[q] && !((taken >> q) & 1u) ? order_key(v[q]) : 0;
            if (o > key) {
                key = o;
                at = 64 * q + lane;
            }
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            const uint32_t ok2 = __shfl_xor(key, d);
            const int at2 = __shfl_xor(at, d);
            if (ok2 > key || (ok2 == key && at2 < at)) {
                key = ok2;
                at = at2;
            }
        }
        if (key == 0) break;
        if ((at & 63) == lane) taken |= 1u << (at >> 6);
        const float val = __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
        if (j == 0) top = val;
        if (lane == j) {
            mine = val;
            my_id = at;
        }
    }
    float p = 0.f;
    if (sigmoid) {
        if (my_id >= 0) p = 1.f / (1.f + expf(-mine));
    } else {
        // exp(l - top), 1 where l == top (also at +inf)
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (ok[q]) sum += v[q] == top ? 1.f : expf(v[q] - top);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
        if (my_id >= 0) p = (mine == top ? 1.f : expf(mine - top)) / sum;
    }
    if (renormalise) {
        float sum = p;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
        if (sum > 0.f) p /= sum;
    }
    if (lane < k) {
        ids[t * k + lane] = my_id;
        w[t * k + lane] = my_id >= 0 ? p * scale : 0.f;
    }
}

// ------------------------------------------------------------------ expert layer

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kDownPairs = 512;  // pairs of one moe_down workgroup

// The pairs of the experts chosen by `n` places of ids, grouped by expert:
// active expert a (in index order) is act[a], its pairs list[off[a] .. off[a+1]).
template <int MAXP> struct ExpertLists {
    int cursor[kMoeMaxExperts];
    uint16_t act[kMoeMaxExperts];
    uint16_t off[kMoeMaxExperts + 1];
    uint16_t list[MAXP];
    int n_act;

    // All threads of the workgroup; ends with a barrier.  Places whose id is no
    // expert are left out.  (The order of one expert's pairs may differ from run
    // to run; each pair is a column of its own in every product, so no result
    // depends on it.)
    __device__ void build(const int32_t *ids, int n, int experts, int threads) {
        const int tid = threadIdx.x, lane = tid & 63;
        for (int e = tid; e < experts; e += threads) cursor[e] = 0;
        __syncthreads();
        for (int p = tid; p < n; p += threads) {
            const int e = ids[p];
            if (e >= 0 && e < experts) atomicAdd(&cursor[e], 1);
        }
        __syncthreads();
        if (tid < 64) {
            int base = 0, na = 0;
            for (int e0 = 0; e0 < experts; e0 += 64) {
                const int e = e0 + lane;
                const int c = e < experts ? cursor[e] : 0;
                int incl = c;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int v = __shfl_up(incl, d);
                    if (lane >= d) incl += v;
                }
                const uint64_t m = __ballot(c > 0);
                if (c > 0) {
                    const int a = na + __popcll(m & ((uint64_t{1} << lane) - 1));
                    act[a] = (uint16_t)e;
                    off[a] = (uint16_t)(base + incl - c);
                }
                if (e < experts) cursor[e] = base + incl - c;
                base += __shfl(incl, 63);
                na += __popcll(m);
            }
            if (lane == 0) {
                off[na] = (uint16_t)base;
                n_act = na;
            }
        }
        __syncthreads();
        for (int p = tid; p < n; p += threads) {
            const int e = ids[p];
            if (e >= 0 && e < experts) list[atomicAdd(&cursor[e], 1)] = (uint16_t)p;
        }
        __syncthreads();
    }
};

// One group of at most 16 TN pairs of an expert: partial sums of the
// wavefronts' K ranges, joined in LDS, then H.
template <typename E, int TN>
__device__ __forceinline__ void up_group(const MoeArgs<E> &a, const E *const (&w)[2], const uint16_t *pairs, int n,
                                         int64_t f0, float (*red)[4][64][4]) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const E *x[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const int p = pairs[std::min(16 * t + i16, n - 1)];
        x[t] = a.X + (int64_t)(p / a.k) * a.ldx + 8 * g;
    }
    f32x4 acc[2][TN] = {};
    const int steps = (int)((a.c + 31) / 32), per = (steps + kWaves - 1) / kWaves;
    const int s0 = std::min(steps, wave * per), s1 = std::min(steps, s0 + per);
    skinny_product<E, 2, TN, 4>(w, x, a.c, s0, s1, acc);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < TN; ++t) *reinterpret_cast<f32x4 *>(red[wave][m * TN + t][lane]) = acc[m][t];
    __syncthreads();
    for (int u = tid; u < 64 * TN; u += kThreads) {
        const int t = u / 64, l = u % 64, at = 16 * t + (l & 15);
        const int64_t c = f0 + 4 * (l >> 4);
        if (at >= n || c >= a.f) continue;
        f32x4 z[2] = {};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int v = 0; v < kWaves; ++v) z[m] += *reinterpret_cast<const f32x4 *>(red[v][m * TN + t][l]);
        float y[4] = {z[0][0], z[0][1], z[0][2], z[0][3]};
        activate<sizeof(E) == 4>(y, a.act);
#pragma unroll
        for (int q = 0; q < 4; ++q) a.H[(int64_t)pairs[at] * a.f + c + q] = to_elem<E>(y[q] * z[1][q]);
    }
    __syncthreads();
}

template <typename E> __global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs<E> a) {
    __shared__ ExpertLists<kMoeMaxPairs> L;
    __shared__ float red[kWaves][4][64][4];
    L.build(a.ids, a.T * a.k, a.experts, kThreads);
    const int slot = (int)blockIdx.y;
    if (slot >= L.n_act) return;
    const int lane = threadIdx.x & 63;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t fr = std::min<int64_t>(f0 + (lane & 15), a.f - 1);
    const int64_t row = ((int64_t)L.act[slot] * a.f + fr) * a.c + 8 * (lane >> 4);
    const E *w[2] = {a.Wg + row, a.Wu + row};
    for (int p = L.off[slot], e = L.off[slot + 1]; p < e;) {
        if (e - p <= 16) {
            up_group<E, 1>(a, w, L.list + p, e - p, f0, red);
            p += 16;
        } else {
            up_group<E, 2>(a, w, L.list + p, std::min(32, e - p), f0, red);
            p += 32;
        }
    }
}

// A workgroup owns 16 output features of a chunk of tokens.  Its wavefronts
// take (expert, part of f) units; the products of a pair go to the pair's own
// place of P, and the places of a token are added at the end in order.
template <typename E> __global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs<E> a, int chunk, int parts) {
    __shared__ ExpertLists<kDownPairs> L;
    extern __shared__ __align__(16) float P[];  // [parts][chunk k][16]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int t0 = (int)blockIdx.y * chunk, tn = std::min(chunk, a.T - t0);
    const int np = chunk * a.k;
    const int64_t c0 = (int64_t)blockIdx.x * 16;
    L.build(a.ids + (int64_t)t0 * a.k, tn * a.k, a.experts, kThreads);
    const int steps = (int)((a.f + 31) / 32), per = (steps + parts - 1) / parts;
    const int64_t cr = std::min<int64_t>(c0 + i16, a.c - 1);
    for (int u = wave; u < L.n_act * parts; u += kWaves) {
        const int s = u / parts, part = u % parts;
        const int s0 = std::min(steps, part * per), s1 = std::min(steps, s0 + per);
        const E *w[1] = {a.Wd + ((int64_t)L.act[s] * a.c + cr) * a.f + 8 * g};
        for (int p = L.off[s], e = L.off[s + 1]; p < e; p += 16) {
            const int pair = L.list[std::min(p + i16, e - 1)];
            const E *x[1] = {a.H + ((int64_t)t0 * a.k + pair) * a.f + 8 * g};
            f32x4 acc[1][1] = {};
            skinny_product<E, 1, 1, 8>(w, x, a.f, s0, s1, acc);
            if (p + i16 < e) *reinterpret_cast<f32x4 *>(P + ((int64_t)part * np + pair) * 16 + 4 * g) = acc[0][0];
        }
    }
    __syncthreads();
    for (int u = tid; u < tn * 16; u += kThreads) {
        const int t = u / 16, q = u % 16;
        const int64_t tok = t0 + t;
        if (c0 + q >= a.c) continue;
        float y = a.R ? to_f32(a.R[tok * a.ldr + c0 + q]) : 0.f, sum = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int e = a.ids[tok * a.k + j];
            if (e < 0 || e >= a.experts) continue;
            float o = 0.f;
            for (int s = 0; s < parts; ++s) o += P[((int64_t)s * np + t * a.k + j) * 16 + q];
            sum += a.w[tok * a.k + j] * o;
        }
        a.Y[tok * a.ldy + c0 + q] = to_elem<E>(sum + y);
    }
}

}  // namespace

template <typename E>
hipError_t launch_route(const E *logits, int64_t ld, int64_t T, int En, int k, bool sigmoid, bool renormalise,
                        float scale, int32_t *ids, float *w, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    const int64_t grid = (T + 3) / 4;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
#define DYRA_ROUTE(P)                                                                                              \
    hipLaunchKernelGGL((route_kernel<E, P>), dim3((unsigned)grid), dim3(256), 0, st, logits, ld, T, En, k, sigmoid, \
                       renormalise, scale, ids, w)
    if (En <= 64) DYRA_ROUTE(1);
    else if (En <= 128) DYRA_ROUTE(2);
    else if (En <= 256) DYRA_ROUTE(4);
    else if (En <= 512) DYRA_ROUTE(8);
    else DYRA_ROUTE(16);
#undef DYRA_ROUTE
    return hipGetLastError();
}

template <typename E> hipError_t launch_moe(const MoeArgs<E> &a, hipStream_t st) {
    if (a.T <= 0) return hipSuccess;
    const int pairs = a.T * a.k;
    if (pairs > kMoeMaxPairs || a.experts > kMoeMaxExperts) return hipErrorInvalidValue;
    const int slots = std::min(a.experts, pairs);
    hipLaunchKernelGGL((moe_up_kernel<E>), dim3((unsigned)((a.f + 15) / 16), (unsigned)slots), dim3(kThreads), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int chunk = std::min(a.T, kDownPairs / a.k);
    // units enough for two rounds of the wavefronts, within 32 KB of partial sums
    const int parts = std::max(1, std::min({(2 * kWaves + slots - 1) / slots, kDownPairs / (chunk * a.k),
                                            (int)((a.f + 255) / 256)}));
    hipLaunchKernelGGL((moe_down_kernel<E>),
                       dim3((unsigned)((a.c + 15) / 16), (unsigned)((a.T + chunk - 1) / chunk)), dim3(kThreads),
                       sizeof(float) * (size_t)parts * chunk * a.k * 16, st, a, chunk, parts);
    return hipGetLastError();
}

template hipError_t launch_route<float>(const float *, int64_t, int64_t, int, int, bool, bool, float, int32_t *, float *,
                                        hipStream_t);
template hipError_t launch_route<bf16>(const bf16 *, int64_t, int64_t, int, int, bool, bool, float, int32_t *, float *,
                                       hipStream_t);
template hipError_t launch_moe<float>(const MoeArgs<float> &, hipStream_t);
template hipError_t launch_moe<bf16>(const MoeArgs<bf16> &, hipStream_t);

}  // namespace dyra
