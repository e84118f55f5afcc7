// What the large tiles of 8-bit operands end with: scales and biases, loaded ahead of a
// tile's products, and the epilogue on a wavefront's sums of 16 TB tokens x 64 weight rows (64
// features, or 32 gate and the same 32 up rows).
#pragma once

#include "ffn_tile.h"
#include "gelu_table.h"

namespace dyra {

template <int N> using ic = std::integral_constant<int, N>;

__device__ __forceinline__ unsigned bits_of(bf16 v) { return __builtin_bit_cast(unsigned short, v); }
__device__ __forceinline__ unsigned bits_of(float v) { return __builtin_bit_cast(unsigned, v); }
template <typename T> __device__ __forceinline__ float value_of(unsigned bits) {
    return __builtin_bit_cast(float, sizeof(T) == 2 ? bits << 16 : bits);
}

// Lane l holds the scale and the bias of the wavefront's weight row l, and the scales of its
// tokens l and 64 + l: loaded before a tile's products, which leave them time to arrive.
// Loaded in the epilogue, one after the other, they cost it 2 us a tile.
template <typename O, bool GATED> struct TileScales {
    float w, x[2];
    unsigned bias;
    // `row` the wavefront's first token, `col` its first feature
    __device__ __forceinline__ void load(const LinearArgs<i8, O> &a, int row, int col, int l) {
        const bool up = GATED && l >= 32;
        const unsigned f = (unsigned)min(col + (GATED ? l & 31 : l), (int)a.N - 1);
        w = (up ? a.scale.w1 : a.scale.w0)[f];
        bias = 0;
        const O *const b = up ? a.b1 : a.b0;
        if (b) bias = bits_of(b[f]);
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = a.scale.x[(unsigned)min(row + 64 * h + l, (int)a.M - 1)];
    }
};

// The epilogue.  `row` and `col` as above, `el` the lane, `mine` 512 bytes of LDS of the wavefront,
// `table` the workgroup's GeluTable (bf16 results with kActGelu); `whole`: no token or feature
// lies past the end.
template <int TB, bool GATED, typename O>
__device__ __forceinline__ void scaled_epilogue(const LinearArgs<i8, O> &a, const i32x4 (&acc)[2][2][4][2], TileScales<O, GATED> s,
                                                float *mine, const char *table, int64_t row0, int64_t col0, int el, bool whole) {
    constexpr int HW = GATED ? 1 : 2;
    const int ei = el & 15, eg = el >> 4;
    const int64_t c = col0 + 8 * eg;  // hw = 1: 32 on
    // Rows whose residual is in flight together: what registers allow.  A row's is asked for
    // before the row FIT ahead of it is stored, as a wait for loads waits for older stores, and
    // the first ones before the sums are scaled, where that spills no registers.  us, FIT rows
    // at a time | this: 25728 x 1024 -> 4096 173 | 163, with GELU 178 | 171, 25728 x 4096 -> 1024
    // 111 | 109, 16384 x 14336 -> 4096 704 | 694.
    constexpr int FIT = (TB == 8 ? 2 : 4) * 2 / (int)sizeof(O);
    constexpr bool EARLY = TB < 8;
    const int64_t first = row0 + ei, step = 16 * a.ldy, step_r = 16 * a.ldr;
    Residual8<O> res[FIT][HW];
    int64_t at_r = 0;
    auto request = [&](int i) __attribute__((always_inline)) {
        asm volatile("" : "+v"(at_r));  // no addresses of later rows are held
#pragma unroll
        for (int hw = 0; hw < HW; ++hw) res[i % FIT][hw].request(a.R + at_r + 32 * hw);
        at_r += step_r;
    };
    auto request_first = [&]() __attribute__((always_inline)) {
        at_r = first * a.ldr + c;
#pragma unroll
        for (int i = 0; i < FIT; ++i) request(i);
    };
    if (!GATED && EARLY && whole && a.R) request_first();
    // Results before the activation, in the sums' registers, all made here: left to the
    // activations' copies of the code, the compiler made them ahead of the branch all the
    // same, and kept 46 to 172 registers in scratch.
    f32x4 z[2][2][4][2];
    asm volatile("" : "+v"(s.bias));  // no conversion, and no wait for it, ahead of the products
    mine[el] = s.x[0];
    mine[64 + el] = s.x[1];
    float sx[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) sx[i] = mine[16 * i + ei];
    __builtin_amdgcn_wave_barrier();
    mine[el] = s.w;  // a wavefront's LDS accesses are in order
    mine[64 + el] = value_of<O>(s.bias);
#pragma unroll
    for (int hw = 0; hw < 2; ++hw)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x4 sw = *reinterpret_cast<const f32x4 *>(mine + 32 * hw + 8 * eg + 4 * j);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(mine + 64 + 32 * hw + 8 * eg + 4 * j);
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                f32x4 &v = z[i >> 2][hw][i & 3][j];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = biased(acc[i >> 2][hw][i & 3][j][q], sx[i], sw[q], b[q]);
                asm volatile("" : "+v"(v));
            }
        }
    __builtin_amdgcn_sched_barrier(0);
    // ACT below 0: of the call, with guards
    auto finish = [&](auto act, auto residual) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        constexpr bool RESIDUAL = decltype(residual)::value;
        int64_t at = first * a.ldy + c;
        if constexpr (RESIDUAL && ACT >= 0 && !EARLY) request_first();
        // both halves of a row one after the other: whole 128-byte lines
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            asm volatile("" : "+v"(at));
            if (ACT < 0 && first + 16 * i >= a.M) break;
            float v[HW][8];
#pragma unroll
            for (int hw = 0; hw < HW; ++hw) {
                f32x4(&s)[2] = z[i >> 2][hw][i & 3];
                if (ACT >= 0) asm volatile("" : "+v"(s[0]), "+v"(s[1]));  // nothing of it is made ahead of the branches
#pragma unroll
                for (int q = 0; q < 8; ++q) v[hw][q] = s[q >> 2][q & 3];
                const int kind = ACT >= 0 ? ACT : a.act;
                if (sizeof(O) == 2 && kind == kActGelu) gelu_from<ACT >= 0 ? 8 : 1>(table, v[hw]);
                else activate<sizeof(O) == 4>(v[hw], kind);
                if constexpr (GATED) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[hw][q] *= z[i >> 2][1][i & 3][q >> 2][q & 3];
                }
                // The activation's last product and this addition would make one FMA here, where ACT is
                // known, and in no kernel that asks for it at run time: other bits.
                if constexpr (RESIDUAL && ACT >= 0) res[i % FIT][hw].add_rounded(v[hw]);
            }
            if constexpr (RESIDUAL && ACT >= 0) {
                if (i + FIT < TB) request(i + FIT);
            }
#pragma unroll
            for (int hw = 0; hw < HW; ++hw) {
                const int have = ACT >= 0 ? 8 : (int)max((int64_t)0, min((int64_t)8, a.N - c - 32 * hw));
                if constexpr (RESIDUAL && ACT < 0) add_row(v[hw], a.R + (first + 16 * i) * a.ldr + c + 32 * hw, have);
                // Past the L2 where the residual's rows go through it too: 16384 x 14336 -> 4096
                // 711 us without, 698 with, others 0 to 1 %.  Without a residual a tile waits
                // longer for its stores: 16384 x 2048 -> 8192 259 us without, 301 with.
                store_row<RESIDUAL && ACT >= 0>(a.Y + at + 32 * hw, v[hw], have);
            }
            at += step;
            if (RESIDUAL || i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // every row: 1 to 2 % without a residual
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
}

}  // namespace dyra
