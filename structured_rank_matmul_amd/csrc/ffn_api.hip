// C entry points of the feed-forward operators: argument checks, then one
// launcher.  Nothing is enqueued unless every check passes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "../../include/dyra.h"
#include "ffn_kernels.h"

namespace {

using dyra::bf16;

// Tokens, output features: the launches of any such sizes whose outputs fit the
// card have less than 2^32 threads.
constexpr int64_t kMaxDim = int64_t{1} << 25;
// Elements of a row of X or of a weight, and between rows: the kernels address
// the rows of a tile by 32-bit byte offsets from its first.
constexpr int64_t kMaxRow = int64_t{1} << 20;
// The same for the expert layer, whose pairs' rows (at most kMoeMaxPairs) are all
// addressed from the first.
constexpr int64_t kMaxExpertRow = int64_t{1} << 18;
dyra_status hip_status(hipError_t e) { return e == hipSuccess ? DYRA_OK : DYRA_ERR_HIP; }
bool aligned(const void *p, size_t n) { return (uintptr_t)p % n == 0; }
bool known(dyra_dtype t) { return t == DYRA_BF16 || t == DYRA_F32; }
size_t size_of(dyra_dtype t) { return t == DYRA_BF16 ? 2 : 4; }
bool known_act(dyra_act a) { return a >= DYRA_ACT_NONE && a <= DYRA_ACT_SILU; }

// Whether an output (not null) is at the address of one of these.
bool among(const void *out, std::initializer_list<const void *> inputs) {
    for (const void *p : inputs)
        if (p == out) return true;
    return false;
}
// Whether Y of several rows is a residual whose rows lie otherwise.
bool other_rows(const void *Y, int64_t ldy, int64_t N, const void *R, int64_t ldr) { return R == Y && N > 1 && ldr != ldy; }

// The checks that the linear layer and the gated pair share.  DYRA_OK with
// *empty set: nothing to do.
dyra_status check_linear(const void *X, int64_t ldx, const void *W0, const void *W1, int64_t ldw, int64_t N, int64_t c1,
                         int64_t c2, dyra_dtype dtype, const void *b0, const void *b1, dyra_act act, const void *Y,
                         int64_t ldy, dyra_dtype out, bool *empty) {
    *empty = false;
    if (!known(dtype) || !known(out) || (dtype == DYRA_F32 && out != DYRA_F32)) return DYRA_ERR_DTYPE;
    if (!known_act(act)) return DYRA_ERR_ARG;
    if (N < 0 || c1 <= 0 || c2 <= 0 || N > kMaxDim || c2 > kMaxDim) return DYRA_ERR_SHAPE;
    if (c1 > kMaxRow || ldx > kMaxRow || ldw > kMaxRow) return DYRA_ERR_SHAPE;
    const int64_t vec = 16 / (int64_t)size_of(dtype);
    if (c1 % vec != 0) return DYRA_ERR_SHAPE;
    if (ldx < c1 || ldw < c1 || ldy < c2) return DYRA_ERR_ARG;
    if (ldx % vec != 0 || ldw % vec != 0) return DYRA_ERR_ALIGN;
    if (N == 0) {
        *empty = true;
        return DYRA_OK;
    }
    if (!X || !W0 || !W1 || !Y) return DYRA_ERR_ARG;
    if (!aligned(X, 16) || !aligned(W0, 16) || !aligned(W1, 16)) return DYRA_ERR_ALIGN;
    if (!aligned(Y, size_of(out)) || !aligned(b0, size_of(dtype)) || !aligned(b1, size_of(dtype))) return DYRA_ERR_ALIGN;
    return DYRA_OK;
}

template <typename E, typename O, bool GATED> dyra_status run(const dyra::LinearArgs<E, O> &a, hipStream_t st) {
    if (a.M <= dyra::kSkinnyTokens) return hip_status(dyra::launch_skinny<E, O, GATED>(a, st));
    if (dyra::takes_narrow(sizeof(E), GATED, a.M, a.N)) return hip_status(dyra::launch_narrow<E, O, GATED>(a, st));
    return hip_status(dyra::launch_linear<E, O, GATED>(a, st));
}

template <typename E, typename O, bool GATED>
dyra_status run_linear(const void *X, int64_t ldx, const void *W0, const void *W1, int64_t ldw, int64_t N, int64_t c1,
                       int64_t c2, const void *b0, const void *b1, dyra_act act, const void *R, int64_t ldr, void *Y,
                       int64_t ldy, void *stream) {
    const dyra::LinearArgs<E, O> a{(const E *)X,  ldx, (const E *)W0, (const E *)W1, ldw, N, c2, c1,
                                   (const E *)b0, (const E *)b1, (const O *)R,   ldr, (O *)Y, ldy, (int)act};
    return run<E, O, GATED>(a, (hipStream_t)stream);
}

}  // namespace

extern "C" {

dyra_status dyra_linear(const void *X, int64_t ldx, const void *Wt, int64_t ldw, int64_t N, int64_t c1, int64_t c2,
                        dyra_dtype dtype, const void *bias, dyra_act act, const void *residual, int64_t ldr,
                        dyra_dtype out_dtype, void *Y, int64_t ldy, void *stream) {
    bool empty;
    const dyra_status s = check_linear(X, ldx, Wt, Wt, ldw, N, c1, c2, dtype, bias, nullptr, act, Y, ldy, out_dtype, &empty);
    if (s != DYRA_OK) return s;
    if (residual && ldr != 0 && ldr < c2) return DYRA_ERR_ARG;
    if (empty) return DYRA_OK;
    if (!aligned(residual, size_of(out_dtype))) return DYRA_ERR_ALIGN;
    if (among(Y, {X, Wt, bias}) || other_rows(Y, ldy, N, residual, ldr)) return DYRA_ERR_ARG;
    if (!residual) ldr = 0;
    if (dtype == DYRA_F32)
        return run_linear<float, float, false>(X, ldx, Wt, nullptr, ldw, N, c1, c2, bias, nullptr, act, residual, ldr, Y, ldy, stream);
    if (out_dtype == DYRA_F32)
        return run_linear<bf16, float, false>(X, ldx, Wt, nullptr, ldw, N, c1, c2, bias, nullptr, act, residual, ldr, Y, ldy, stream);
    return run_linear<bf16, bf16, false>(X, ldx, Wt, nullptr, ldw, N, c1, c2, bias, nullptr, act, residual, ldr, Y, ldy, stream);
}

dyra_status dyra_gated(const void *X, int64_t ldx, const void *Wg, const void *Wu, int64_t ldw, int64_t N, int64_t c1,
                       int64_t c2, dyra_dtype dtype, const void *bias_g, const void *bias_u, dyra_act act, void *H,
                       int64_t ldh, void *stream) {
    bool empty;
    const dyra_status s = check_linear(X, ldx, Wg, Wu, ldw, N, c1, c2, dtype, bias_g, bias_u, act, H, ldh, dtype, &empty);
    if (s != DYRA_OK || empty) return s;
    if (among(H, {X, Wg, Wu, bias_g, bias_u})) return DYRA_ERR_ARG;
    if (dtype == DYRA_F32)
        return run_linear<float, float, true>(X, ldx, Wg, Wu, ldw, N, c1, c2, bias_g, bias_u, act, nullptr, 0, H, ldh, stream);
    return run_linear<bf16, bf16, true>(X, ldx, Wg, Wu, ldw, N, c1, c2, bias_g, bias_u, act, nullptr, 0, H, ldh, stream);
}

dyra_status dyra_route(const void *logits, int64_t ld, int64_t T, int32_t experts, int32_t topk, dyra_dtype dtype,
                       dyra_score score, int32_t renormalise, float scale, int32_t *ids, float *weights, void *stream) {
    if (!known(dtype)) return DYRA_ERR_DTYPE;
    if (score != DYRA_SCORE_SOFTMAX && score != DYRA_SCORE_SIGMOID) return DYRA_ERR_ARG;
    if (!std::isfinite(scale)) return DYRA_ERR_ARG;
    if (T < 0 || T > kMaxDim || experts < 1 || experts > dyra::kMoeMaxExperts) return DYRA_ERR_SHAPE;
    if (topk < 1 || topk > experts || topk > 64) return DYRA_ERR_SHAPE;
    if (ld < experts) return DYRA_ERR_ARG;
    if (T == 0) return DYRA_OK;
    if (!logits || !ids || !weights) return DYRA_ERR_ARG;
    if (!aligned(logits, size_of(dtype)) || !aligned(ids, 4) || !aligned(weights, 4)) return DYRA_ERR_ALIGN;
    if (among(ids, {logits, weights}) || among(weights, {logits})) return DYRA_ERR_ARG;
    hipStream_t st = (hipStream_t)stream;
    const bool sg = score == DYRA_SCORE_SIGMOID, rn = renormalise != 0;
    if (dtype == DYRA_BF16)
        return hip_status(dyra::launch_route<bf16>((const bf16 *)logits, ld, T, experts, topk, sg, rn, scale, ids, weights, st));
    return hip_status(dyra::launch_route<float>((const float *)logits, ld, T, experts, topk, sg, rn, scale, ids, weights, st));
}

size_t dyra_moe_workspace_bytes(int64_t T, int32_t topk, int64_t f, dyra_dtype dtype) {
    if (T < 0 || topk < 1 || topk > 64 || f < 1 || f > kMaxExpertRow || T > dyra::kMoeMaxPairs / topk || !known(dtype)) return 0;
    if (f % (16 / (int64_t)size_of(dtype)) != 0) return 0;
    return (size_t)T * (size_t)topk * (size_t)f * size_of(dtype);
}

dyra_status dyra_moe(const void *X, int64_t ldx, int64_t T, int64_t c, int64_t f, const void *Wg, const void *Wu,
                     const void *Wd, int32_t experts, const int32_t *ids, const float *weights, int32_t topk,
                     dyra_dtype dtype, dyra_act act, const void *residual, int64_t ldr, void *Y, int64_t ldy,
                     void *workspace, size_t workspace_bytes, void *stream) {
    if (!known(dtype)) return DYRA_ERR_DTYPE;
    if (!known_act(act)) return DYRA_ERR_ARG;
    const int64_t vec = 16 / (int64_t)size_of(dtype);
    if (T < 0 || c < 1 || f < 1 || c % vec != 0 || f % vec != 0) return DYRA_ERR_SHAPE;
    if (c > kMaxExpertRow || f > kMaxExpertRow || ldx > kMaxExpertRow) return DYRA_ERR_SHAPE;
    if (experts < 1 || experts > dyra::kMoeMaxExperts || topk < 1 || topk > 64) return DYRA_ERR_SHAPE;
    if (T > dyra::kMoeMaxPairs / topk) return DYRA_ERR_SHAPE;
    if (ldx < c || ldy < c || (residual && ldr != 0 && ldr < c)) return DYRA_ERR_ARG;
    if (ldx % vec != 0) return DYRA_ERR_ALIGN;
    if (T == 0) return DYRA_OK;
    if (!X || !Wg || !Wu || !Wd || !ids || !weights || !Y) return DYRA_ERR_ARG;
    if (!aligned(X, 16) || !aligned(Wg, 16) || !aligned(Wu, 16) || !aligned(Wd, 16)) return DYRA_ERR_ALIGN;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(Y, size_of(dtype)) || !aligned(residual, size_of(dtype)))
        return DYRA_ERR_ALIGN;
    if (!workspace || workspace_bytes < dyra_moe_workspace_bytes(T, topk, f, dtype)) return DYRA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return DYRA_ERR_ALIGN;
    // Y over X is fine: X is read for the last time before Y is first written
    if (among(Y, {Wg, Wu, Wd, ids, weights}) || other_rows(Y, ldy, T, residual, ldr)) return DYRA_ERR_ARG;
    if (among(workspace, {Y, X, Wg, Wu, Wd, ids, weights, residual})) return DYRA_ERR_ARG;
    const size_t inner = dyra_moe_workspace_bytes(T, topk, f, dtype);
    // what is there beyond the inner activations: room for split sums, then for what
    // the activations' rounding leaves out
    const size_t split = (size_t)T * dyra::kMoePartBytes;
    const bool rest = dtype == DYRA_BF16 && workspace_bytes >= 2 * inner + split;
    float *const parts = workspace_bytes >= inner + split ? (float *)((char *)workspace + (rest ? 2 : 1) * inner) : nullptr;
    hipStream_t st = (hipStream_t)stream;
    auto go = [&](auto e) {
        typedef decltype(e) E;
        const dyra::MoeArgs<E> a{(const E *)X, ldx, (const E *)Wg, (const E *)Wu, (const E *)Wd, ids, weights, c, f,
                                 (int)T, topk, experts, (int)act, (const E *)residual, residual ? ldr : 0, (E *)Y, ldy,
                                 (E *)workspace, rest, parts};
        return hip_status(dyra::launch_moe<E>(a, st));
    };
    return dtype == DYRA_BF16 ? go(bf16{}) : go(float{});
}

}  // extern "C"
