// 256 x 256 tiles (224 and 192 x 256 too) of the linear layer and the gated pair, bf16, for products
// that fill the chip: eight wavefronts in two groups of four that take turns on
// the matrix cores.
//
// A workgroup owns 32 TB tokens and 256 weight rows (256 output features, or 128
// gate and the same 128 up rows).  Wavefront (wm, wn) owns TB blocks of 16 tokens
// (4 in half A, the rest in half B) and 64 weight rows: 16 TB accumulator
// registers.  TB is 8; 7 and 6 serve products that the lower tiles divide into
// fewer or smaller rounds of one tile per CU (their panel keeps 128 rows per wm,
// the last ones empty).  K advances in slabs of 64 (128
// bytes per row) through two LDS buffers.  A slab is two phases, one per half of
// the wavefront's tokens, 32 MFMAs each:
//
//     phase  reads into registers                    product            copies
//     0      tokens A (8 x 16 B), weights B (4)       A x weights A, B   tokens B of slab s + 1, weights A of s + 2
//     1      tokens B (8), weights A of s + 1 (4)     B x weights A, B   tokens A, weights B of slab s + 2
//
// The kernel is persistent and the copies run on through the end of a tile: the
// last two slabs of a tile copy the first two of the workgroup's next one (of
// its last tile, one more time the first two of that), so a tile's epilogue
// falls between two slabs of an unbroken stream.  K is taken to a whole number
// of slab pairs; what lies past K is zero in LDS, by the buffer load's range
// check.
//
// A phase is [reads, copies, waits] barrier [MFMAs] barrier, and the second
// group (wm = 1, sharing each SIMD with the first) runs one barrier behind, so
// that one group's 512 cycles of MFMAs cover the other's reads (about 400 at
// 128 bytes a cycle).  Every read is waited for before the barrier that ends its
// half of the phase, so a region may be copied over one phase after its last
// read.  A copy has two phases (a slab) to land: each phase waits until at most
// 8 newer copies are outstanding, and the barrier after it publishes them.  A
// wavefront's stores count among its copies and complete in order with them; up
// to the first copy issued after an epilogue, the waits leave that epilogue's
// stores outstanding too (when their number is known: whole tiles).
//
// Four phases of 16 MFMAs a slab, one per quadrant, took 811 us at 8192^3 where
// two of 32 take 730 (1.51 PFLOP/s; the library's product 680).
#pragma once

#include "ffn_tile.h"

namespace dyra {

template <int N> using ic = std::integral_constant<int, N>;

// The lane number, computed anew: what is derived from it is not kept in
// registers across the main loop (whose accumulators and fragments need them).
__device__ __forceinline__ int fresh_lane() {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    return l;
}

template <typename O, bool GATED, int TB>
__global__ __launch_bounds__(512, 2) void linear_big_kernel(LinearArgs<bf16, O> a, int tiles_m, int tiles_n,
                                                            int per_xcd) {
    constexpr int BM = 32 * TB, BF = GATED ? 128 : 256;
    constexpr int STAGE = 32768, WOFF = 65536;  // two buffers of 256 token rows of 128 bytes, two of 256 weight rows
    // 16-byte stores of a wavefront's epilogue
    constexpr int STORES = (GATED ? 1 : 2) * TB * (8 * (int)sizeof(O) / 16);
    __shared__ __align__(16) char smem[4 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int i16 = lane & 15, g = lane >> 4;
    // XCD x works on a contiguous band of tiles, one after the other on its
    // workgroups.  Within the band, tiles run down groups of 8 token rows, so
    // that the 32 tiles an XCD holds at a time are 8 x 4 and share their
    // operands' slabs in its L2.
    const int ntiles = tiles_m * tiles_n, nslots = (int)(gridDim.x / 8);
    const int band = (int)(blockIdx.x % 8) * per_xcd, band_end = min(band + per_xcd, ntiles);
    int tile = band + (int)(blockIdx.x / 8);
    if (tile >= band_end) return;
    auto place = [&](int t, int64_t &row0, int64_t &col0) {
        const int group = t / (8 * tiles_n), in_group = t - group * 8 * tiles_n;
        const int gm = min(tiles_m - 8 * group, 8);
        row0 = (int64_t)(8 * group + in_group % gm) * BM;
        col0 = (int64_t)(in_group / gm) * BF;
    };

    // This lane's part of the copies: wavefront w copies the 1 KB blocks w and
    // w + 8 of each region (8 rows of 128 bytes; lane l fills position l % 8 of
    // row l / 8 with the chunk that the row's swizzle puts there).  A region's
    // rows: tokens 64 half .. + 63 of both wm, weights 32 half .. + 31 of every
    // wn.  Rows past the end are read from the last row.
    uint32_t xoff[2][2], woff[2][2];  // [half][block], bytes from the tile's first row
    __amdgpu_buffer_rsrc_t xbuf, wbuf0, wbuf1;
    const int xchunk = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
    const int wchunk = 16 * ((lane & 7) ^ (((lane >> 4) & 1) | ((wave & 3) << 1)));
    auto sources = [&](int64_t row0, int64_t col0) __attribute__((always_inline)) {
        xbuf = panel(a.X + row0 * a.ldx);
        wbuf0 = panel(a.W0 + col0 * a.ldw);
        if constexpr (GATED) wbuf1 = panel(a.W1 + col0 * a.ldw);
        const int tmax = (int)min(a.M - 1 - row0, (int64_t)BM - 1), fmax = (int)min(a.N - 1 - col0, (int64_t)BF - 1);
        const int lr = fresh_lane() >> 3;
        const uint32_t xld = (uint32_t)(2 * a.ldx), wld = (uint32_t)(2 * a.ldw);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = 64 * h + 8 * wave + lr;  // of the 128 that the panel has for wm = q
                xoff[h][q] = r < 16 * TB ? (uint32_t)min(16 * TB * q + r, tmax) * xld + xchunk : kOutside;
                const int b = wave + 8 * q;
                const int f = (GATED ? 32 : 64) * (b >> 2) + (GATED ? 0 : 32 * h) + 8 * (b & 3) + lr;
                woff[h][q] = (uint32_t)min(f, fmax) * wld + wchunk;
            }
    };
    const int slabs = 2 * (int)((a.K + 127) / 128);
    // the slab that the copies are at: its bytes left in a row, its buffer
    int cs = 0, left = (int)min((int64_t)INT32_MAX, 2 * a.K);
    const int row_bytes = left;
    auto copy_x = [&](int h, int buf) __attribute__((always_inline)) {
        char *dst = smem + buf * STAGE + (64 * h + 8 * wave) * 128;
        const bool in = xchunk < left;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            buffer_to_lds16(xbuf, in ? xoff[h][q] : kOutside, 128 * cs, dst + q * 128 * 128);
    };
    auto copy_w = [&](int h, int buf) __attribute__((always_inline)) {
        char *dst = smem + buf * STAGE + WOFF + (64 * (wave >> 2) + 32 * h + 8 * (wave & 3)) * 128;
        const bool in = wchunk < left;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            buffer_to_lds16(GATED && h ? wbuf1 : wbuf0, in ? woff[h][q] : kOutside, 128 * cs, dst + q * 128 * 128);
    };
    int64_t row0, col0;            // of the tile being computed
    int64_t next_row0, next_col0;  // of the tile being copied
    auto advance = [&](bool switches) __attribute__((always_inline)) {  // the copies' next slab
        ++cs;
        left -= 128;
        if (switches && cs == slabs) {
            cs = 0;
            left = row_bytes;
            const int t = tile + nslots;
            if (t < band_end) {
                place(t, next_row0, next_col0);
                sources(next_row0, next_col0);
            }
        }
    };

    f32x4 acc[2][2][4][2];  // [token half][weight half][token block][weight block]
    bf16x8 fx[2][4];        // [32-deep step][token block]
    bf16x8 fw[3][2][2];     // [slot][step][weight block]

    const int swx = (i16 >> 1) & 7, sww = ((i16 >> 1) & 1) | ((i16 >> 2) << 1);
    const char *const px = smem + (128 * wm + i16) * 128;
    const char *const pw = smem + WOFF + (64 * wn + 8 * (i16 >> 2) + (i16 & 3)) * 128;
    auto read_x = [&](int h, int buf) __attribute__((always_inline)) {
        const char *p = px + buf * STAGE + 64 * h * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < (h == 0 ? 4 : TB - 4); ++i)
                fx[k][i] = *reinterpret_cast<const bf16x8 *>(p + 16 * i * 128 + (((4 * k + g) ^ swx) << 4));
    };
    auto read_w = [&](int h, int buf, int slot) __attribute__((always_inline)) {
        const char *p = pw + buf * STAGE + 32 * h * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fw[slot][k][j] = *reinterpret_cast<const bf16x8 *>(p + 4 * j * 128 + (((4 * k + g) ^ sww) << 4));
    };
    // 32 MFMAs: token half hx with both weight halves
    auto products = [&](int hx, int slot_a, int slot_b) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        barrier_only();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int hw = 0; hw < 2; ++hw)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < (hx == 0 ? 4 : TB - 4); ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[hx][hw][i][j] = mma32(acc[hx][hw][i][j], fw[hw ? slot_b : slot_a][k][j], fx[k][i]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        barrier_only();
    };
    bool stores_out = false;  // the stores of the last epilogue may be left outstanding
    auto landed = [&](bool early) __attribute__((always_inline)) {
        if (early) wait_lds_and_vm<8 + STORES>();
        else wait_lds_and_vm<8>();
    };
    // One slab in buffer B; slot B holds weights A.
    auto slab = [&](auto buffer, bool early) __attribute__((always_inline)) {
        constexpr int B = decltype(buffer)::value;
        read_x(0, B);
        read_w(1, B, 2);
        copy_x(1, 1 - B);
        advance(B == 0);  // an even number of slabs: the copies change tiles in slab 0 of a pair
        copy_w(0, B);
        landed(early && B == 0);
        products(0, B, 2);
        read_x(1, B);
        read_w(0, 1 - B, 1 - B);
        copy_x(0, B);
        copy_w(1, B);
        landed(early && B == 0);
        products(1, B, 2);
    };

    place(tile, row0, col0);
    next_row0 = row0;
    next_col0 = col0;
    sources(row0, col0);
    copy_w(0, 0);
    copy_x(0, 0);
    copy_w(1, 0);
    copy_x(1, 0);
    advance(false);
    copy_w(0, 1);
    copy_x(0, 1);
    copy_w(1, 1);
    wait_vmcnt<8>();
    barrier_only();
    read_w(0, 0, 0);
    wait_lds_and_vm<8>();
    barrier_only();
    if (wm == 1) barrier_only();
    for (;;) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            f32x4 z = {};
            asm volatile("" : "+v"(z));  // plain zeroed registers: no first iteration of its own
            acc[i >> 4][(i >> 3) & 1][(i >> 1) & 3][i & 1] = z;
        }
#pragma clang loop unroll(disable)
        for (int s = 0; s < slabs; s += 2) {
            slab(ic<0>{}, stores_out);
            slab(ic<1>{}, stores_out);
            stores_out = false;
        }
        // ---- epilogue: 8 consecutive features of a token per pair of weight blocks.
        // Whole tiles run a copy of the code made for their activation, without
        // guards. One copy for everything, with branches over what a call does not
        // use, took 181 us (no epilogue) and 195 us (bias and residual) at 25728 x
        // 4096 -> 1024; this takes 175 and 187 (the library's bare product 169).
        const int el = fresh_lane(), ei = el & 15, eg = el >> 4;
        const bool whole = row0 + BM <= a.M && col0 + BF <= a.N;
        stores_out = whole;
        constexpr int HW = GATED ? 1 : 2;
        const int64_t c = col0 + (GATED ? 32 : 64) * wn + 8 * eg;  // hw = 1: 32 on
        float b0[HW][8] = {}, b1[8] = {};
#pragma unroll
        for (int hw = 0; hw < HW; ++hw)
            if (a.b0) load_row(a.b0 + c + 32 * hw, b0[hw], whole ? 8 : (int)(a.N - c) - 32 * hw);
        if (GATED && a.b1) load_row(a.b1 + c, b1, whole ? 8 : (int)(a.N - c));
        // ACT below 0: of the call, with guards
        auto finish = [&](auto act, auto residual) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            constexpr bool RESIDUAL = decltype(residual)::value;
            // rows whose residual is in flight together: what registers allow
            constexpr int BATCH = RESIDUAL && ACT >= 0 ? (TB == 8 ? 2 : 4) * 2 / (int)sizeof(O) : 1;
            const int64_t first = row0 + 16 * TB * wm + ei;
            // both halves of a row one after the other: whole 128-byte lines
#pragma unroll
            for (int i0 = 0; i0 < TB; i0 += BATCH) {
                Residual8<O> r[BATCH][HW];
                if constexpr (RESIDUAL && ACT >= 0) {
#pragma unroll
                    for (int i = i0; i < i0 + BATCH && i < TB; ++i)
#pragma unroll
                        for (int hw = 0; hw < HW; ++hw) r[i - i0][hw].request(a.R + (first + 16 * i) * a.ldr + c + 32 * hw);
                }
#pragma unroll
                for (int i = i0; i < i0 + BATCH && i < TB; ++i) {
                    const int64_t t = first + 16 * i;
                    if (ACT < 0 && t >= a.M) continue;
#pragma unroll
                    for (int hw = 0; hw < HW; ++hw) {
                        const int have = ACT >= 0 ? 8 : (int)max((int64_t)0, min((int64_t)8, a.N - c - 32 * hw));
                        float v[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = acc[i >> 2][hw][i & 3][q >> 2][q & 3] + b0[hw][q];
                        activate<sizeof(O) == 4>(v, ACT >= 0 ? ACT : a.act);
                        if constexpr (GATED) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) v[q] *= acc[i >> 2][1][i & 3][q >> 2][q & 3] + b1[q];
                        }
                        if constexpr (RESIDUAL && ACT >= 0) r[i - i0][hw].add_to(v);
                        else if constexpr (RESIDUAL) add_row(v, a.R + t * a.ldr + c + 32 * hw, have);
                        store_row(a.Y + t * a.ldy + c + 32 * hw, v, have);
                    }
                }
            }
        };
        auto finish_act = [&](auto act) __attribute__((always_inline)) {
            if constexpr (!GATED) {
                if (a.R) return finish(act, std::true_type{});
            }
            finish(act, std::false_type{});
        };
        if (!whole) finish_act(ic<-1>{});
        else if (a.act == kActNone) finish_act(ic<kActNone>{});
        else if (a.act == kActRelu) finish_act(ic<kActRelu>{});
        else if (a.act == kActGelu) finish_act(ic<kActGelu>{});
        else if (a.act == kActGeluTanh) finish_act(ic<kActGeluTanh>{});
        else finish_act(ic<kActSilu>{});
        tile += nslots;
        if (tile >= band_end) break;
        row0 = next_row0;
        col0 = next_col0;
    }
    if (wm == 0) barrier_only();
    wait_vmcnt<0>();  // no copy may land in LDS after the workgroup has given it back
}

template <typename O, bool GATED, int TB> hipError_t launch_big(const LinearArgs<bf16, O> &a, hipStream_t st) {
    const int64_t tiles_m = (a.M + 32 * TB - 1) / (32 * TB), tiles_n = (a.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    const int64_t ntiles = tiles_m * tiles_n;
    if (ntiles > (int64_t)1 << 24) return hipErrorInvalidValue;
    const int64_t per_xcd = (ntiles + 7) / 8;
    // one workgroup per CU: 32 on each XCD
    const int64_t slots = per_xcd < 32 ? per_xcd : 32;
    hipLaunchKernelGGL((linear_big_kernel<O, GATED, TB>), dim3((unsigned)(8 * slots)), dim3(512), 0, st, a, (int)tiles_m,
                       (int)tiles_n, (int)per_xcd);
    return hipGetLastError();
}

}  // namespace dyra
