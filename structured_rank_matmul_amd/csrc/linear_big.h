// 256 x 256 tiles of the linear layer and the gated pair, bf16, for products
// that fill the chip: eight wavefronts in two groups of four that take turns on
// the matrix cores.
//
// A workgroup owns 256 tokens and 256 weight rows (256 output features, or 128
// gate and the same 128 up rows).  Wavefront (wm, wn) owns tokens 128 wm .. and
// 64 weight rows: 128 accumulator registers.  K advances in slabs of 64 (128
// bytes per row) through two LDS buffers.  A slab is four phases, one per
// quadrant (token half x weight half) of the wavefront's block, 16 MFMAs each:
//
//     phase   reads into registers       product         copies
//     0       tokens A (8 x 16 B)         A x weights A   tokens B of slab s + 1
//     1       weights B (4)               A x weights B   weights A of slab s + 2
//     2       tokens B (8)                B x weights B   tokens A of slab s + 2
//     3       weights A of slab s + 1 (4) B x weights A   weights B of slab s + 2
//
// A phase is [reads, copies, wait] barrier [MFMAs] barrier, and the second
// group (wm = 1, sharing each SIMD with the first) runs one barrier behind, so
// that one group's MFMAs cover the other's reads.  A region of a buffer is
// copied over two phases after its last read was issued: the read has then been
// waited for by MFMAs that every wavefront finished a barrier before.  A copy
// has five phases to land: each phase waits until at most 10 newer copies are
// outstanding, and the barrier after it publishes them.
#pragma once

#include "ffn_tile.h"

namespace dyra {

template <int N> using ic = std::integral_constant<int, N>;

template <typename O, bool GATED>
__global__ __launch_bounds__(512, 2) void linear_big_kernel(LinearArgs<bf16, O> a, int tiles_m, int tiles_n,
                                                            int per_xcd) {
    constexpr int BM = 256, BF = GATED ? 128 : 256;
    constexpr int STAGE = 65536, WOFF = 32768;  // a buffer: 256 token rows, then 256 weight rows, of 128 bytes
    __shared__ __align__(16) char smem[2 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    // XCD x works on a contiguous band of tiles; within it, tiles run down
    // groups of 8 token rows, so that the 32 tiles an XCD holds at a time are
    // 8 x 4 and share their operands' slabs in its L2
    const int idx = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
    if (idx >= tiles_m * tiles_n) return;
    const int group = idx / (8 * tiles_n), in_group = idx - group * 8 * tiles_n;
    const int gm = tiles_m - 8 * group < 8 ? tiles_m - 8 * group : 8;
    const int64_t row0 = (int64_t)(8 * group + in_group % gm) * BM;
    const int64_t col0 = (int64_t)(in_group / gm) * BF;

    // This lane's part of the copies: wavefront w copies the 1 KB blocks w and
    // w + 8 of each region (8 rows of 128 bytes; lane l fills position l % 8 of
    // row l / 8 with the chunk that the row's swizzle puts there).
    // A region's rows: tokens 64 half .. + 63 of both wm, weights 32 half .. +
    // 31 of every wn.  Rows past the end are read from the last row.
    uint32_t xoff[2][2], woff[2][2];  // [half][block]
    const char *const xbase = reinterpret_cast<const char *>(a.X + row0 * a.ldx);
    const char *const wbase0 = reinterpret_cast<const char *>(a.W0 + col0 * a.ldw);
    const char *const wbase1 = reinterpret_cast<const char *>((GATED ? a.W1 : a.W0) + col0 * a.ldw);
    const int lr = lane >> 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int rx = 128 * q + 64 * h + 8 * wave + lr;
            const int64_t tx = row0 + rx < a.M ? rx : a.M - 1 - row0;
            xoff[h][q] = (uint32_t)(tx * a.ldx * 2) + 16 * ((lane & 7) ^ ((rx >> 1) & 7));
            const int b = wave + 8 * q;
            const int rw = 64 * (b >> 2) + 32 * h + 8 * (b & 3) + lr;               // row of the panel
            const int fw = GATED ? 32 * (b >> 2) + 8 * (b & 3) + lr : rw;           // feature of the tile
            const int64_t tw = col0 + fw < a.N ? fw : a.N - 1 - col0;
            woff[h][q] = (uint32_t)(tw * a.ldw * 2) + 16 * ((lane & 7) ^ (((rw >> 1) & 1) | (((rw >> 3) & 3) << 1)));
        }
    const int slabs = (int)((a.K + 63) / 64);
    const int rem = (int)(a.K - (int64_t)(slabs - 1) * 64) * 2;  // bytes of the last slab's rows
    // the chunks past the end of a partial last slab are fetched from its first
    // one; their products are masked when it is read
    auto copy_x = [&](int s, int h) __attribute__((always_inline)) {
        char *dst = smem + (s & 1) * STAGE + (64 * h + 8 * wave) * 128;
        const char *base = xbase + (int64_t)s * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t o = xoff[h][q];
            if (s == slabs - 1) {
                const int c = (lane & 7) ^ (((8 * wave + lr) >> 1) & 7);
                o -= 16 * c < rem ? 0 : 16 * c;
            }
            lds_dma16(base + o, dst + q * 128 * 128);
        }
    };
    auto copy_w = [&](int s, int h) __attribute__((always_inline)) {
        char *dst = smem + (s & 1) * STAGE + WOFF;
        const char *base = (GATED && h ? wbase1 : wbase0) + (int64_t)s * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int b = wave + 8 * q;
            uint32_t o = woff[h][q];
            if (s == slabs - 1) {
                const int rw = 8 * (b & 3) + lr;
                const int c = (lane & 7) ^ (((rw >> 1) & 1) | (((rw >> 3) & 3) << 1));
                o -= 16 * c < rem ? 0 : 16 * c;
            }
            lds_dma16(base + o, dst + (64 * (b >> 2) + 32 * h + 8 * (b & 3)) * 128);
        }
    };

    f32x4 acc[2][2][4][2];  // [token half][weight half][token block][weight block]
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i >> 4][(i >> 3) & 1][(i >> 1) & 3][i & 1] = f32x4{};
    bf16x8 fx[2][4];        // [32-deep step][token block]
    bf16x8 fw[2][2][2];     // [slot][step][weight block]

    const int swx = (i16 >> 1) & 7, sww = ((i16 >> 1) & 1) | ((i16 >> 2) << 1);
    const char *const px = smem + (128 * wm + i16) * 128;
    const char *const pw = smem + WOFF + (64 * wn + 8 * (i16 >> 2) + (i16 & 3)) * 128;
    auto read_x = [&](int s, int h) __attribute__((always_inline)) {
        const char *p = px + (s & 1) * STAGE + 64 * h * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fx[k][i] = *reinterpret_cast<const bf16x8 *>(p + 16 * i * 128 + (((4 * k + g) ^ swx) << 4));
    };
    auto read_w = [&](int s, int h, int slot) __attribute__((always_inline)) {
        const char *p = pw + (s & 1) * STAGE + 32 * h * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fw[slot][k][j] = *reinterpret_cast<const bf16x8 *>(p + 4 * j * 128 + (((4 * k + g) ^ sww) << 4));
    };
    auto products = [&](int hx, int hw, int slot, bool mask) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        barrier_only();
        if (mask) {  // elements past K: zero in both operands
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if ((4 * k + g) * 16 >= rem) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) fx[k][i] = bf16x8{};
#pragma unroll
                    for (int j = 0; j < 2; ++j) fw[slot][k][j] = bf16x8{};
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[hx][hw][i][j] = mma32(acc[hx][hw][i][j], fw[slot][k][j], fx[k][i]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        barrier_only();
    };
    // One slab; A: the slot that holds weights A.  In the last two slabs fewer
    // copies are outstanding: LAST2 and LAST1 of them are newer than the one the
    // next phase reads.
    auto slab = [&](int s, auto slot_a) __attribute__((always_inline)) {
        constexpr int A = decltype(slot_a)::value, B = 1 - A;
        const int ahead = slabs - 1 - s;  // slabs after this one
        const bool mask = ahead == 0 && rem < 128;
        auto landed = [&](auto last2, auto last1) __attribute__((always_inline)) {
            if (ahead >= 2) wait_vmcnt<10>();
            else if (ahead == 1) wait_vmcnt<decltype(last2)::value>();
            else wait_vmcnt<decltype(last1)::value>();
        };
        read_x(s, 0);
        if (ahead >= 1) copy_x(s + 1, 1);
        landed(ic<10>{}, ic<2>{});
        products(0, 0, A, mask);
        read_w(s, 1, B);
        if (ahead >= 2) copy_w(s + 2, 0);
        landed(ic<8>{}, ic<0>{});
        products(0, 1, B, mask);
        read_x(s, 1);
        if (ahead >= 2) copy_x(s + 2, 0);
        landed(ic<6>{}, ic<0>{});
        products(1, 1, B, mask);
        read_w(s + 1, 0, B);  // past the last slab: a buffer's old bytes, not used
        if (ahead >= 2) copy_w(s + 2, 1);
        landed(ic<4>{}, ic<0>{});
        products(1, 0, A, mask);
    };
    copy_w(0, 0);
    copy_x(0, 0);
    copy_w(0, 1);
    copy_x(0, 1);
    if (slabs > 1) {
        copy_w(1, 0);
        copy_x(1, 0);
        copy_w(1, 1);
        wait_vmcnt<10>();
    } else {
        wait_vmcnt<4>();
    }
    barrier_only();
    read_w(0, 0, 0);
    if (wm == 1) barrier_only();
    for (int s = 0; s < slabs; s += 2) {
        slab(s, ic<0>{});
        if (s + 1 < slabs) slab(s + 1, ic<1>{});
    }
    if (wm == 0) barrier_only();

    // ---- epilogue: 8 consecutive features of a token per pair of weight blocks
#pragma unroll
    for (int hw = 0; hw < (GATED ? 1 : 2); ++hw) {
        const int64_t c = col0 + (GATED ? 32 * wn : 64 * wn + 32 * hw) + 8 * g;
        const int have = (int)(a.N - c < 8 ? a.N - c : 8);
        if (have <= 0) continue;
        float b0[8] = {}, b1[8] = {};
        if (a.b0) load_row(a.b0 + c, b0, false, have);
        if (GATED && a.b1) load_row(a.b1 + c, b1, false, have);
#pragma unroll
        for (int hx = 0; hx < 2; ++hx)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = row0 + 128 * wm + 64 * hx + 16 * i + i16;
                if (t >= a.M) continue;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = acc[hx][hw][i][q >> 2][q & 3] + b0[q];
                activate<sizeof(O) == 4>(v, a.act);
                if constexpr (GATED) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] *= acc[hx][1][i][q >> 2][q & 3] + b1[q];
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

template <typename O, bool GATED> hipError_t launch_big(const LinearArgs<bf16, O> &a, hipStream_t st) {
    const int64_t tiles_m = (a.M + 255) / 256, tiles_n = (a.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    const int64_t ntiles = tiles_m * tiles_n;
    // a tile's operand rows are addressed by 32-bit byte offsets from its first
    if (ntiles > (int64_t)1 << 28 || a.ldx > (int64_t)1 << 22 || a.ldw > (int64_t)1 << 22) return hipErrorInvalidValue;
    const int64_t per_xcd = (ntiles + 7) / 8;
    hipLaunchKernelGGL((linear_big_kernel<O, GATED>), dim3((unsigned)(8 * per_xcd)), dim3(512), 0, st, a, (int)tiles_m,
                       (int)tiles_n, (int)per_xcd);
    return hipGetLastError();
}

}  // namespace dyra
