// Argument blocks and launchers of the feed-forward kernels: the linear layer
// with its epilogue and the gated pair (linear_tile.h for many tokens,
// skinny_linear.h for few), the router and the expert layer (moe.hip), and the
// norm and quantisation of rows (rows.hip).  All enqueue on `st` and return the
// launch status; none allocates or synchronises.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn_choice.h"

namespace dyra {

typedef __bf16 bf16;
typedef int8_t i8;

// Activations, numbered as dyra_act.
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// What goes with the operands of a product: the type of its biases, and, of 8-bit
// integers, the scale of every token and of every weight row.
template <typename E, typename O> struct Operands {
    typedef E Bias;
    struct Scales {
        static constexpr const float *x = nullptr, *w0 = nullptr, *w1 = nullptr;
    };
};
template <typename O> struct Operands<i8, O> {
    typedef O Bias;
    struct Scales {
        const float *x, *w0, *w1;  // [M], [N], [N] or null
    };
};

// One linear layer (W1 null) or gated pair (W1 not null), E operands, O output.
//   linear: Y = act(X W0^T + b0) + R       gated: Y = act(X W0^T + b0) * (X W1^T + b1)
// Of 8-bit integers the products are scaled: scale.x_i scale.w_j sum_k X_ik W_jk.
template <typename E, typename O> struct LinearArgs {
    typedef typename Operands<E, O>::Bias Bias;
    const E *X;
    int64_t ldx;
    const E *W0, *W1;  // [N][K] each, rows ldw elements apart
    int64_t ldw;
    int64_t M, N, K;   // tokens, output features, input features (K a multiple of 16 / sizeof(E))
    const Bias *b0, *b1;  // [N] or null
    const O *R;        // [M][N], rows ldr apart, or null
    int64_t ldr;
    O *Y;              // [M][N], rows ldy apart
    int64_t ldy;
    int act;
    typename Operands<E, O>::Scales scale;
};

template <typename E, typename O, bool GATED> hipError_t launch_linear(const LinearArgs<E, O> &a, hipStream_t st);
// 8-bit operands with K in parts (s.parts > 1): split_bytes() of `work`.
template <typename O, bool GATED>
hipError_t launch_split(const LinearArgs<i8, O> &a, const Split &s, int32_t *work, hipStream_t st);
// Few tokens: the weights are streamed once.
template <typename E, typename O, bool GATED> hipError_t launch_skinny(const LinearArgs<E, O> &a, hipStream_t st);
// Few features (up to 32, gated 16) of many tokens: X is streamed.
template <typename E, typename O, bool GATED> hipError_t launch_narrow(const LinearArgs<E, O> &a, hipStream_t st);

// Router: the k largest of every row of logits.
template <typename E>
hipError_t launch_route(const E *logits, int64_t ld, int64_t T, int E_n, int k, bool sigmoid, bool renormalise,
                        float scale, int32_t *ids, float *w, hipStream_t st);

// Expert layer: Y[t] = R[t] + sum_j w[t][j] FFN_{ids[t][j]}(X[t]).
template <typename E> struct MoeArgs {
    const E *X;
    int64_t ldx;
    const E *Wg, *Wu;  // [experts][f][c]
    const E *Wd;       // [experts][c][f]
    const int32_t *ids;
    const float *w;    // [T][k]
    int64_t c, f;
    int T, k, experts;
    int act;
    const E *R;
    int64_t ldr;
    E *Y;
    int64_t ldy;
    E *H;              // [T k][f], workspace; with `rest` [T k][f / 8][2][8]
    bool rest;         // of every 8 features what their rounding left out follows (bf16)
    float *parts;      // kMoePartBytes a token, workspace, or null
};
template <typename E> hipError_t launch_moe(const MoeArgs<E> &a, hipStream_t st);

// Root-mean-square norm of rows (W null: ones), E rows; Y of E or, in 8 bits with a
// scale for each row, of i8:
//   z = X + R,  S = z,  Y = z / sqrt(mean z^2 + eps) * W
// launch_quantize makes 8-bit rows of X alone: y = X.
template <typename E> struct RowArgs {
    const E *X;
    int64_t ldx;
    const E *R;        // [N][c], rows ldr apart, or null
    int64_t ldr;
    const E *W;        // [c] or null
    int64_t N, c;
    float eps;
    E *S;              // [N][c], rows lds apart, or null
    int64_t lds;
    void *Y;           // [N][c], rows ldy apart
    int64_t ldy;
    float *scales;     // [N], of 8-bit rows
};
template <typename E> hipError_t launch_norm(const RowArgs<E> &a, hipStream_t st);
template <typename E> hipError_t launch_norm_quantize(const RowArgs<E> &a, hipStream_t st);
template <typename E> hipError_t launch_quantize(const RowArgs<E> &a, hipStream_t st);
template <typename E>
hipError_t launch_dequantize(const i8 *Q, int64_t ldq, const float *scales, int64_t N, int64_t c, E *X, int64_t ldx,
                             hipStream_t st);

}  // namespace dyra
