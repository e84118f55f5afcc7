// Linear layer and gated pair for more tokens than skinny.hip takes:
//     Y = act(X W^T + b) + R           H = act(X Wg^T + bg) * (X Wu^T + bu)
// one pass over X and the weights, the epilogue applied to the accumulators.
// Products that fill the chip with 256 x 256 tiles take linear_big.h's kernel;
// the tiles here, from 32 x 64 to 128 x 256, are for those that would not.
//
// A workgroup owns BM tokens x BF output features (gated: BF features of both
// products, so a lane holds a feature's gate and up sums together and the
// pair never reaches memory).  K advances in stages of SL slabs of 128 bytes per
// row, copied from global memory straight into LDS, NS stages in flight (for bf16
// 100 to 144 KB: with one tile per CU, depth is what hides the latency), one
// barrier per stage.  A slab row is 8 chunks of 16 bytes, chunk c at position c ^ sw(row), so
// that the 16 rows a 16-lane group reads fall on distinct banks; the swizzle is
// applied by choosing which chunk each lane of the copy fetches.  Rows past the
// end, chunks past K and stages past the last are read out of the buffers'
// range: zeros, and one wait fits every stage.
//
// Output layout: the weights are the first MFMA operand, so a lane's registers
// run along output features.  Rows of the weight panel are dealt to pairs of
// 16 x 16 blocks so that the pair's 8 registers are 8 consecutive features
// (block q, row i holds feature 8 (i / 4) + 4 q + i % 4 of the pair's 32): the
// epilogue stores 16 bytes per lane straight from registers, 64 bytes of a row
// per instruction, with no pass through LDS.
//
// Small tiles are bound by reading their fragments from LDS (a 64 x 128 slab: 64
// KB by eight wavefronts of 32 x 32).  So the wavefronts form KS groups that take
// the 32-deep steps in turn on larger parts of the tile (64 x 64: 32 KB), and add
// their sums through LDS at the end: bf16 slabs of 32 x 64, 64 x 64, 64 x 128, 128 x
// 128 and 128 x 256 tiles take 149, 179, 291, 498 and 830 ns where one group of
// smaller parts took 163, 194, 349, 549 and 913.  (Operands in the L2s; from memory see
// ffn_choice.h.)
#include "linear_big.h"

#include <algorithm>
#include <cmath>

namespace dyra {

namespace {

template <typename E, int BM, int BF, int WM, int WN, int KS, int NS, int SL, bool GATED> struct TileShape {
    static constexpr int NW = WM * WN * KS;
    static constexpr int BN = GATED ? 2 * BF : BF;   // rows of the weight panel
    static constexpr int TM = BM / WM / 16;          // token blocks of a wavefront
    static constexpr int TF = BF / WN / 16;          // feature blocks of a wavefront (per product)
    static constexpr int TN = GATED ? 2 * TF : TF;
    static constexpr int PER_WAVE = (BM + BN) / 8 / NW;  // 1 KB copies of a slab
    static constexpr int SLAB = (BM + BN) * 128, STAGE = SL * SLAB;
    static_assert((BM + BN) / 8 % NW == 0 && BM / 8 % NW == 0 && BF / 8 % NW == 0, "whole copies per panel");
    static constexpr int PER_CU = NS * STAGE <= 80 * 1024 ? 2 : 1;  // workgroups
    static constexpr int STEPS = SL * 4 / (int)sizeof(E);  // 32-deep steps of a stage
    static constexpr int OWNERS = KS < TM ? KS : TM;  // K groups that finish token blocks
    static_assert(STEPS % KS == 0 && TM % OWNERS == 0, "whole steps for each K group, token blocks for each owner");
    static_assert((KS - 1) * TM * TN * 1024 * WM * WN <= NS * STAGE, "room for the K groups' sums");
    static_assert(TF % 2 == 0 && TM >= 1 && BF % 32 == 0 && NS * STAGE <= 160 * 1024, "tile shape");
};

template <typename E, typename O, int BM, int BF, int WM, int WN, int KS, int NS, int SL, bool GATED>
__global__ __launch_bounds__(64 * WM * WN * KS, (TileShape<E, BM, BF, WM, WN, KS, NS, SL, GATED>::PER_CU * WM * WN * KS / 4)) void
linear_tile_kernel(LinearArgs<E, O> a, int tiles_n, int ntiles, int per_xcd) {
    using S = TileShape<E, BM, BF, WM, WN, KS, NS, SL, GATED>;
    __shared__ __align__(16) char smem[NS * S::STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;  // K group, place in the tile
    const int i16 = lane & 15, g = lane >> 4;
    // workgroup ids are dealt round-robin over the 8 XCDs; each XCD walks a
    // contiguous band of tiles, down the tokens first, so tiles that share
    // weights share an L2
    const int tile = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
    if (tile >= ntiles) return;
    const int tiles_m = ntiles / tiles_n;
    const int64_t row0 = (int64_t)(tile % tiles_m) * BM;
    const int64_t col0 = (int64_t)(tile / tiles_m) * BF;

    // this wavefront's copies of a slab: block q of 8 rows, BM / 8 / NW of them
    // tokens, the rest weights (gate rows, then up rows)
    constexpr int XQ = BM / 8 / S::NW, FQ = BF / 8 / S::NW;
    const auto bytes_from = [&](int64_t rows, int64_t from, int64_t ld) {
        return ((rows - 1 - from) * ld + a.K) * (int64_t)sizeof(E);
    };
    const __amdgpu_buffer_rsrc_t xbuf = panel(a.X + row0 * a.ldx, bytes_from(a.M, row0, a.ldx));
    const __amdgpu_buffer_rsrc_t w0buf = panel(a.W0 + col0 * a.ldw, bytes_from(a.N, col0, a.ldw));
    const __amdgpu_buffer_rsrc_t w1buf = GATED ? panel(a.W1 + col0 * a.ldw, bytes_from(a.N, col0, a.ldw)) : w0buf;
    uint32_t off[S::PER_WAVE], chunk[S::PER_WAVE];
#pragma unroll
    for (int q = 0; q < S::PER_WAVE; ++q) {
        const int r = 8 * (wave + q * S::NW) + (lane >> 3);  // panel row
        if (q < XQ) {
            chunk[q] = 16 * ((lane & 7) ^ ((r >> 1) & 7));
            off[q] = (uint32_t)r * (uint32_t)(a.ldx * sizeof(E)) + chunk[q];
        } else {
            const int rw = r - BM, f = q < XQ + FQ ? rw : rw - BF;
            chunk[q] = 16 * ((lane & 7) ^ (((rw >> 1) & 1) | (((rw >> 3) & 3) << 1)));
            off[q] = (uint32_t)f * (uint32_t)(a.ldw * sizeof(E)) + chunk[q];
        }
    }
    const int row_bytes = (int)(a.K * (int64_t)sizeof(E));
    const int stages = (row_bytes + 128 * SL - 1) / (128 * SL);
    auto issue = [&](int s) __attribute__((always_inline)) {
        char *dst = smem + s % NS * S::STAGE;
#pragma unroll
        for (int h = 0; h < SL; ++h) {
            const int k = (s * SL + h) * 128, left = row_bytes - k;
#pragma unroll
            for (int q = 0; q < S::PER_WAVE; ++q)
                buffer_to_lds16(q < XQ ? xbuf : q < XQ + FQ ? w0buf : w1buf, (int)chunk[q] < left ? off[q] : kOutside,
                                left > 0 ? (uint32_t)k : 0u, dst + h * S::SLAB + (wave + q * S::NW) * 1024);
        }
    };

    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) acc[i][j] = f32x4{};

#pragma unroll
    for (int p = 0; p < NS - 1; ++p) issue(p);
    const int swx = (i16 >> 1) & 7, sww = ((i16 >> 1) & 1) | ((i16 >> 2) << 1);
    const int wrow = 8 * (i16 >> 2) + (i16 & 3);
    for (int s = 0; s < stages; ++s) {
        // all but the stages issued after s have landed; the barrier makes every
        // wavefront's part visible and frees the buffer of stage s - 1
        wait_vmcnt<(NS - 2) * SL * S::PER_WAVE>();
        barrier_only();
        issue(s + NS - 1);
        const char *sx = smem + s % NS * S::STAGE + (wm * S::TM * 16 + i16) * 128;
        const char *sw = smem + s % NS * S::STAGE + (BM + wn * S::TF * 16 + wrow) * 128;
        typedef typename Frag<E>::type F;
        auto frag = [&](const char *row, int h, int swz) -> F {
            if constexpr (sizeof(E) == 2) {
                return *reinterpret_cast<const bf16x8 *>(row + (((4 * h + g) ^ swz) << 4));
            } else {
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(row + ((g ^ swz) << 4));
                const f32x4 hi = *reinterpret_cast<const f32x4 *>(row + (((4 + g) ^ swz) << 4));
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        };
        constexpr int PER_SLAB = 4 / (int)sizeof(E);  // steps of a slab
#pragma unroll
        for (int step = 0; step < S::STEPS / KS; ++step) {
            const int hh = KS * step + kg, slab = hh / PER_SLAB * S::SLAB, h = hh % PER_SLAB;
            F fw[S::TN], fx[S::TM];
#pragma unroll
            for (int j = 0; j < S::TN; ++j) {
                const int jf = j % S::TF;
                fw[j] = frag(sw + slab + ((j / S::TF) * BF + 32 * (jf >> 1) + 4 * (jf & 1)) * 128, h, sww);
            }
#pragma unroll
            for (int i = 0; i < S::TM; ++i) fx[i] = frag(sx + slab + i * 16 * 128, h, swx);
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int j = 0; j < S::TN; ++j) acc[i][j] = mma32(acc[i][j], fw[j], fx[i]);
        }
    }
    wait_vmcnt<0>();  // no copy may land in LDS after the workgroup has given it back
    // ---- the K groups' sums: group q finishes token blocks q, q + OWNERS, ..
    constexpr int OWN = S::TM / S::OWNERS;
    f32x4 sum[OWN][S::TN];
    if constexpr (KS == 1) {
#pragma unroll
        for (int i = 0; i < OWN; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j) sum[i][j] = acc[i][j];
    } else {
        barrier_only();  // every wavefront is done with the stages
        // [tile place][token block][giving group, the owner left out][weight block][lane]
        auto place = [&](int block, int giver) {
            return smem + ((((wm * WN + wn) * S::TM + block) * (KS - 1) + giver) * S::TN * 64 + lane) * 16;
        };
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int owner = i % S::OWNERS;
            if (owner == kg) {
#pragma unroll
                for (int j = 0; j < S::TN; ++j) sum[i / S::OWNERS][j] = acc[i][j];
            } else {
                char *const p = place(i, kg - (kg > owner));
#pragma unroll
                for (int j = 0; j < S::TN; ++j) *reinterpret_cast<f32x4 *>(p + j * 1024) = acc[i][j];
            }
        }
        __syncthreads();
        if (kg >= S::OWNERS) return;
#pragma unroll
        for (int i = 0; i < OWN; ++i)
#pragma unroll
            for (int o = 0; o < KS - 1; ++o)
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
                    sum[i][j] += *reinterpret_cast<const f32x4 *>(place(kg + S::OWNERS * i, o) + j * 1024);
    }
    // ---- epilogue: 8 consecutive features of one token per pair of blocks
#pragma unroll
    for (int p = 0; p < S::TF / 2; ++p) {
        const int64_t c = col0 + wn * S::TF * 16 + 32 * p + 8 * g;
        const int have = (int)std::min<int64_t>(8, a.N - c);
        if (have <= 0) continue;
        float b0[8] = {}, b1[8] = {};
        if (a.b0) load_row(a.b0 + c, b0, have);
        if (GATED && a.b1) load_row(a.b1 + c, b1, have);
        const bool ahead = !GATED && a.R && have >= 8;
        Residual8<O> r[OWN];
        if (ahead) {
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                r[i].request(a.R + std::min<int64_t>(row0 + (wm * S::TM + S::OWNERS * i + kg) * 16 + i16, a.M - 1) * a.ldr + c);
        }
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int64_t t = row0 + (wm * S::TM + S::OWNERS * i + kg) * 16 + i16;
            if (t >= a.M) continue;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = sum[i][2 * p + (q >> 2)][q & 3] + b0[q];
            activate<sizeof(O) == 4>(v, a.act);
            if constexpr (GATED) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= sum[i][S::TF + 2 * p + (q >> 2)][q & 3] + b1[q];
            } else if (ahead) {
                r[i].add_to(v);
            } else if (a.R) {
                add_row(v, a.R + t * a.ldr + c, have);
            }
            store_row(a.Y + t * a.ldy + c, v, have);
        }
    }
}

template <typename E, typename O, int BM, int BF, int WM, int WN, int KS, int NS, int SL, bool GATED>
hipError_t launch_tile(const LinearArgs<E, O> &a, hipStream_t st) {
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BF - 1) / BF;
    const int64_t ntiles = tiles_m * tiles_n;
    if (ntiles > (int64_t)INT32_MAX - 8) return hipErrorInvalidValue;
    const int64_t per_xcd = (ntiles + 7) / 8;
    hipLaunchKernelGGL((linear_tile_kernel<E, O, BM, BF, WM, WN, KS, NS, SL, GATED>), dim3((unsigned)(8 * per_xcd)),
                       dim3(64 * WM * WN * KS), 0, st, a, (int)tiles_n, (int)ntiles, (int)per_xcd);
    return hipGetLastError();
}

}  // namespace

template <typename E, typename O, bool GATED> hipError_t launch_linear(const LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    const Tile tile = pick_tile(sizeof(E), GATED, a.M, a.N, a.K * (int64_t)sizeof(E));
    if constexpr (sizeof(E) == 2) {
        if (tile == T256x256) return launch_big<O, GATED, 8>(a, st);
        if (tile == T224x256) return launch_big<O, GATED, 7>(a, st);
        if (tile == T192x256) return launch_big<O, GATED, 6>(a, st);
        switch (tile) {
        case T32x64: return launch_tile<E, O, 32, GATED ? 32 : 64, 1, GATED ? 1 : 2, GATED ? 4 : 2, 5, 2, GATED>(a, st);
        case T64x64: return launch_tile<E, O, 64, GATED ? 32 : 64, 1, GATED ? 1 : 2, 4, 4, 2, GATED>(a, st);
        case T64x128: return launch_tile<E, O, 64, GATED ? 64 : 128, 1, 2, 4, 3, 2, GATED>(a, st);
        case T128x128: return launch_tile<E, O, 128, GATED ? 64 : 128, 2, 2, 2, 4, 1, GATED>(a, st);
        default: return launch_tile<E, O, 128, GATED ? 128 : 256, 2, 2, 2, 3, 1, GATED>(a, st);
        }
    } else {
        // Float32 is bound by its MFMAs (eight a step where bf16 has one): fewer stages
        // and two workgroups a CU, one's products over the other's waits (12608 x 768 ->
        // 3000: 561 us with one, 475 with two; the library's product 484).
        switch (tile) {
        case T32x64: return launch_tile<E, O, 32, GATED ? 32 : 64, 2, GATED ? 1 : 2, GATED ? 2 : 1, 5, 2, GATED>(a, st);
        case T64x64: return launch_tile<E, O, 64, GATED ? 32 : 64, 4, GATED ? 1 : 2, 1, 2, 2, GATED>(a, st);
        case T64x128: return launch_tile<E, O, 64, GATED ? 64 : 128, GATED ? 4 : 2, GATED ? 2 : 4, 1, 3, 1, GATED>(a, st);
        default: return launch_tile<E, O, 128, GATED ? 64 : 128, GATED ? 4 : 2, GATED ? 2 : 4, 1, 2, 1, GATED>(a, st);
        }
    }
}

template hipError_t launch_linear<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_linear<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_linear<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
