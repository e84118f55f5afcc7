// Linear layer and gated pair for many tokens:
//     Y = act(X W^T + b) + R           H = act(X Wg^T + bg) * (X Wu^T + bu)
// one pass over X and the weights, the epilogue applied to the accumulators.
//
// A workgroup owns BM tokens x BF output features (gated: BF features of both
// products, so a lane holds a feature's gate and up sums together and the
// pair never reaches memory).  K advances in slices of 128 bytes per row, moved
// from global memory straight into LDS, NS slices in flight, one barrier per
// slice.  A slice row is 8 chunks of 16 bytes, chunk c at position c ^ sw(row),
// so that the 16 rows a 16-lane group reads fall on distinct banks; the swizzle
// is applied by choosing which chunk each lane of the copy fetches.
// A last slice that reaches past K fetches the missing chunks from a zero
// chunk, for both operands.
//
// Output layout: the weights are the first MFMA operand, so a lane's registers
// run along output features.  Rows of the weight panel are dealt to pairs of
// 16 x 16 blocks so that the pair's 8 registers are 8 consecutive features
// (block q, row i holds feature 8 (i / 4) + 4 q + i % 4 of the pair's 32): the
// epilogue stores 16 bytes per lane straight from registers, 64 bytes of a row
// per instruction, with no pass through LDS.
#include "linear_big.h"

#include <algorithm>
#include <cmath>

namespace dyra {

namespace {

__device__ __align__(16) const unsigned g_zero[4] = {0, 0, 0, 0};

template <typename E, int BM, int BF, int WM, int WN, int NS, bool GATED> struct TileShape {
    static constexpr int NW = WM * WN;
    static constexpr int BN = GATED ? 2 * BF : BF;   // rows of the weight panel
    static constexpr int TM = BM / WM / 16;          // token blocks of a wavefront
    static constexpr int TF = BF / WN / 16;          // feature blocks of a wavefront (per product)
    static constexpr int TN = GATED ? 2 * TF : TF;
    static constexpr int BK = 128 / (int)sizeof(E);  // elements of a slice row
    static constexpr int BLOCKS = (BM + BN) / 8;     // 1 KB copies per slice
    static constexpr int PER_WAVE = BLOCKS / NW;
    static constexpr int STAGE = (BM + BN) * 128;
    static_assert(BLOCKS % NW == 0 && TF % 2 == 0 && TM >= 1 && BF % 32 == 0, "tile shape");
};

template <typename E, typename O, int BM, int BF, int WM, int WN, int NS, bool GATED>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile_kernel(LinearArgs<E, O> a, int tiles_n, int ntiles,
                                                                   int per_xcd) {
    using S = TileShape<E, BM, BF, WM, WN, NS, GATED>;
    constexpr int VEC = 16 / (int)sizeof(E);
    __shared__ __align__(16) char smem[NS * S::STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i16 = lane & 15, g = lane >> 4;
    // workgroup ids are dealt round-robin over the 8 XCDs; each XCD walks a
    // contiguous band of tiles, so tiles that share operands share an L2
    const int tile = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
    if (tile >= ntiles) return;
    const int64_t row0 = (int64_t)(tile / tiles_n) * BM;
    const int64_t col0 = (int64_t)(tile % tiles_n) * BF;

    // this wavefront's copies: panel row and chunk per lane (rows past the end
    // are fetched from the last row and never stored)
    const char *src[S::PER_WAVE];
    int chunk[S::PER_WAVE];
#pragma unroll
    for (int q = 0; q < S::PER_WAVE; ++q) {
        const int j = wave + q * S::NW;
        const int r = 8 * j + (lane >> 3);
        if (8 * j < BM) {
            const int64_t t = row0 + r < a.M ? row0 + r : a.M - 1;
            chunk[q] = (lane & 7) ^ ((r >> 1) & 7);
            src[q] = reinterpret_cast<const char *>(a.X + t * a.ldx);
        } else {
            const int rw = r - BM;
            const bool up = GATED && rw >= BF;
            const int64_t n0 = col0 + (up ? rw - BF : rw);
            const int64_t n = n0 < a.N ? n0 : a.N - 1;
            chunk[q] = (lane & 7) ^ (((rw >> 1) & 1) | (((rw >> 3) & 3) << 1));
            src[q] = reinterpret_cast<const char *>((up ? a.W1 : a.W0) + n * a.ldw);
        }
    }
    const int64_t row_bytes = a.K * (int64_t)sizeof(E);
    const int slices = (int)((row_bytes + 127) / 128);
    auto issue = [&](int s) {
        char *dst = smem + (s % NS) * S::STAGE;
        const int64_t off = (int64_t)s * 128;
        const bool whole = off + 128 <= row_bytes;
#pragma unroll
        for (int q = 0; q < S::PER_WAVE; ++q) {
            const int64_t o = off + 16 * chunk[q];
            const void *p = whole || o < row_bytes ? (const void *)(src[q] + o) : (const void *)g_zero;
            lds_dma16(p, dst + (wave + q * S::NW) * 1024);
        }
    };

    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) acc[i][j] = f32x4{};

    for (int p = 0; p < NS - 1 && p < slices; ++p) issue(p);
    const int swx = (i16 >> 1) & 7, sww = ((i16 >> 1) & 1) | ((i16 >> 2) << 1);
    const int wrow = 8 * (i16 >> 2) + (i16 & 3);
    for (int s = 0; s < slices; ++s) {
        // all but the slices issued after s have landed; the barrier makes every
        // wavefront's part visible and frees the buffer of slice s - 1
        if (slices - 1 - s >= NS - 2) wait_vmcnt<(NS - 2) * S::PER_WAVE>();
        else wait_vmcnt<0>();
        barrier_only();
        if (s + NS - 1 < slices) issue(s + NS - 1);
        const char *sx = smem + (s % NS) * S::STAGE + (wm * S::TM * 16 + i16) * 128;
        const char *sw = smem + (s % NS) * S::STAGE + (BM + wn * S::TF * 16 + wrow) * 128;
        typedef typename Frag<E>::type F;
        auto frag = [&](const char *row, int h, int swz) -> F {
            if constexpr (sizeof(E) == 2) {
                return *reinterpret_cast<const bf16x8 *>(row + (((4 * h + g) ^ swz) << 4));
            } else {
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(row + (((2 * g) ^ swz) << 4));
                const f32x4 hi = *reinterpret_cast<const f32x4 *>(row + (((2 * g + 1) ^ swz) << 4));
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        };
#pragma unroll
        for (int h = 0; h < S::BK / 32; ++h) {
            F fw[S::TN], fx[S::TM];
#pragma unroll
            for (int j = 0; j < S::TN; ++j) {
                const int jf = j % S::TF;
                fw[j] = frag(sw + ((j / S::TF) * BF + 32 * (jf >> 1) + 4 * (jf & 1)) * 128, h, sww);
            }
#pragma unroll
            for (int i = 0; i < S::TM; ++i) fx[i] = frag(sx + i * 16 * 128, h, swx);
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int j = 0; j < S::TN; ++j) acc[i][j] = mma32(acc[i][j], fw[j], fx[i]);
        }
    }
    // ---- epilogue: 8 consecutive features of one token per pair of blocks
#pragma unroll
    for (int p = 0; p < S::TF / 2; ++p) {
        const int64_t c = col0 + wn * S::TF * 16 + 32 * p + 8 * g;
        const int have = (int)std::min<int64_t>(8, a.N - c);
        if (have <= 0) continue;
        float b0[8] = {}, b1[8] = {};
        if (a.b0) load_row(a.b0 + c, b0, false, have);
        if (GATED && a.b1) load_row(a.b1 + c, b1, false, have);
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int64_t t = row0 + (wm * S::TM + i) * 16 + i16;
            if (t >= a.M) continue;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = acc[i][2 * p + (q >> 2)][q & 3] + b0[q];
            activate<sizeof(O) == 4>(v, a.act);
            if constexpr (GATED) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= acc[i][S::TF + 2 * p + (q >> 2)][q & 3] + b1[q];
            } else if (a.R) {
                float r[8];
                load_row(a.R + t * a.ldr + c, r, a.vec, have);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += r[q];
            }
            store_row(a.Y + t * a.ldy + c, v, a.vec, have);
        }
    }
}

template <typename E, typename O, int BM, int BF, int WM, int WN, int NS, bool GATED>
hipError_t launch_tile(const LinearArgs<E, O> &a, hipStream_t st) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BF - 1) / BF;
    const int64_t ntiles = tiles_m * tiles_n;
    if (ntiles > (int64_t)INT32_MAX - 8) return hipErrorInvalidValue;
    const int64_t per_xcd = (ntiles + 7) / 8;
    hipLaunchKernelGGL((linear_tile_kernel<E, O, BM, BF, WM, WN, NS, GATED>), dim3((unsigned)(8 * per_xcd)),
                       dim3(64 * WM * WN), 0, st, a, (int)tiles_n, (int)ntiles, (int)per_xcd);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_linear(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    if constexpr (sizeof(E) == 2) {
        const int64_t t256 = ((a.M + 255) / 256) * ((a.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256));
        if (t256 >= 128 && big_strides(a)) return launch_big<O, GATED>(a, st);
    }
    const int64_t big = ((a.M + 127) / 128) * ((a.N + (GATED ? 63 : 127)) / (GATED ? 64 : 128));
    if (big >= 192) return launch_tile<E, O, 128, GATED ? 64 : 128, 2, 2, 2, GATED>(a, st);
    return launch_tile<E, O, 64, GATED ? 32 : 64, 4, 1, 3, GATED>(a, st);
}

template hipError_t launch_linear<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_linear<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_linear<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
