"""Cases of the feed-forward layer in 8-bit integers: the root-mean-square norm
with the residual's addition, quantisation of rows, and the linear layer and the
gated pair of products on integers with a scale for each token and channel.

A case names its operator in "op" and holds plain sizes and choices.  With
``own`` false, ``run`` computes the operator by elementary torch operations in
float32, rounded once at the end; with ``own`` true it calls the library.  Rows
held in 8 bits are returned as the values they stand for, in bfloat16, beside
their scales.
"""
import math

import torch

own = False

OPS_MOST = 3.8e12     # a drawn case costs no more than the largest listed one
VALUES_MOST = 2.3e8   # of a norm or a quantisation

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"
EPS = 1e-5
LEAST = 127.0 * 2.0 ** -126   # the largest magnitude that a row's scale is taken from, at least


# ------------------------------------------------------------------ cases

def norm(name, N, c, dtype="bf16", residual=True, out="i8", pad=0):
    """out: "i8" (values in 8 bits and a scale for each row) or "same".  pad: elements between the rows of X."""
    return {"name": name, "op": "norm", "N": N, "c": c, "dtype": dtype, "residual": residual, "out": out, "pad": pad}


def quantize(name, N, c, dtype="bf16", pad=0):
    return {"name": name, "op": "quantize", "N": N, "c": c, "dtype": dtype, "pad": pad}


def linear(name, N, c1, c2, act="none", bias=False, residual=False, out="bf16", pad=0):
    return {"name": name, "op": "linear", "N": N, "c1": c1, "c2": c2, "act": act, "bias": bias, "residual": residual,
            "out": out, "pad": pad}


def gated(name, N, c1, c2, act="silu", bias=False, out="bf16", pad=0):
    return {"name": name, "op": "gated", "N": N, "c1": c1, "c2": c2, "act": act, "bias": bias, "out": out, "pad": pad}


def listed():
    return [
        # a Llama-style MLP: 8 prompts of 2048 tokens, and one token decoding, from the attention block's output and the
        # residual stream to the gate and up products' 8-bit operand
        norm("norm prefill", 16384, 4096),
        norm("norm one token", 1, 4096),
        # before a ViT-L block that stays in bfloat16: 128 images x 201 tokens
        norm("norm vitl", 25728, 1024, out="same"),
        # float32 rows of an odd length, X a slice of a wider matrix, no residual: one clip's frames and one more
        norm("norm odd f32", 1501, 1003, dtype="f32", residual=False, out="same", pad=5),
        # the MLP's inner activations on their way to the down product: prefill, and 16 sequences decoding
        quantize("quantize prefill", 16384, 14336),
        quantize("quantize decode", 16, 14336),
        # ViT-L fc1 with bias and GELU; the MLP's down product onto the residual stream; a decoding step's projection; a
        # head of an odd number of classes with float32 logits, X a slice of a wider matrix
        linear("vitl fc1 gelu", 25728, 1024, 4096, act="gelu", bias=True),
        linear("down prefill", 16384, 14336, 4096, residual=True),
        linear("one token", 1, 4096, 4096, residual=True),
        linear("odd head", 1501, 1280, 1003, bias=True, out="f32", pad=48),
        # the gate and up products: 8 prompts of 2048 tokens, and 16 sequences decoding
        gated("gated prefill", 16384, 4096, 14336),
        gated("gated decode", 16, 4096, 14336),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "linear", "gated"))
    if op in ("norm", "quantize"):
        c = _between(rng, 1, 16384)
        if rng.random() < 0.6:
            c = -(-c // 64) * 64
        N = _between(rng, 1, min(32768, int(VALUES_MOST / 2 / c) if op == "norm" else int(VALUES_MOST / c)))
        dtype, pad = "f32" if rng.random() < 0.3 else "bf16", rng.choice((0, 0, 0, 5, 64))
        if op == "norm":
            case = norm("", N, c, dtype, rng.random() < 0.6, rng.choice(("i8", "same")), pad)
        else:
            case = quantize("", N, c, dtype, pad)
    else:
        c1, c2 = 16 * _between(rng, 2, 896), _between(rng, 1, 16384)
        if rng.random() < 0.5:
            c2 = -(-c2 // 32) * 32
        N = _between(rng, 1, max(1, min(32768, int(OPS_MOST / ((2.0 if op == "linear" else 4.0) * c1 * c2)))))
        act, bias, out = rng.choice(ACTS), rng.random() < 0.5, "f32" if rng.random() < 0.3 else "bf16"
        pad = rng.choice((0, 0, 0, 16, 208))
        if op == "linear":
            case = linear("", N, c1, c2, act, bias, rng.random() < 0.5, out, pad)
        else:
            case = gated("", N, c1, c2, act, bias, out, pad)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _rows(n, c, gen, dtype, pad=0):
    """Rows with a few large channels, as of a residual stream; a few rows of padding, all zero; pad > 0: a column
    slice of a wider matrix."""
    x = torch.randn(n, c + pad, generator=gen, device=DEVICE)
    x[:, :: max(1, c // 6)] *= 8.0
    if n > 40:
        x[torch.rand(n, generator=gen, device=DEVICE) < 0.02] = 0.0
    return x.to(dtype)[:, pad // 2:][:, :c]


def _inner(n, c, gen, dtype, pad=0):
    """Rows as a gated pair of products gives them: silu(g) u."""
    g = torch.randn(n, c + pad, generator=gen, device=DEVICE)
    return (torch.randn(n, c + pad, generator=gen, device=DEVICE) * g / (1.0 + torch.exp(-g))).to(dtype)[:, pad // 2:][:, :c]


def _eight_bits(shape, gen, spread, pad=0):
    """(int8 values with the row's largest at 127, float32 scales) of rows of normal values."""
    x = torch.randn(shape[0], shape[1] + pad, generator=gen, device=DEVICE)
    a = x.abs().amax(dim=1)
    q = torch.round(x * (127.0 / a)[:, None]).to(torch.int8)[:, pad // 32 * 16:][:, :shape[1]]
    return q, a * (spread / 127.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["X"] = _inner(case["N"], case["c"], gen, TYPES[case["dtype"]], case["pad"])
    elif case["op"] == "norm":
        N, c, t = case["N"], case["c"], TYPES[case["dtype"]]
        s["X"] = _rows(N, c, gen, t, case["pad"])
        s["R"] = (2.0 * torch.randn(N, c, generator=gen, device=DEVICE)).to(t) if case["residual"] else None
        s["w"] = (1.0 + 0.3 * torch.randn(c, generator=gen, device=DEVICE)).to(t)
    else:
        N, c1, c2, o = case["N"], case["c1"], case["c2"], TYPES[case["out"]]
        s["out_type"] = o
        s["X"], s["sx"] = _eight_bits((N, c1), gen, 1.0, case["pad"])
        for n in ("w",) if case["op"] == "linear" else ("g", "u"):
            s["W" + n], s["s" + n] = _eight_bits((c2, c1), gen, c1 ** -0.5)
            s["b" + n] = torch.randn(c2, generator=gen, device=DEVICE).to(o) if case["bias"] else None
        if case["op"] == "linear":
            s["R"] = (2.0 * torch.randn(N, c2, generator=gen, device=DEVICE)).to(o) if case["residual"] else None
    return s


# ------------------------------------------------------------------ one pass

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_eight_bits(y):
    """(values that rows held in 8 bits stand for, scales)."""
    scales = y.abs().amax(dim=1).clamp(min=LEAST) / 127.0
    q = torch.round(y / scales[:, None]).clamp(-127.0, 127.0).to(torch.int8)
    return (q.float() * scales[:, None]).to(torch.bfloat16), scales


def _plain_norm(s):
    z = s["X"].float()
    if s["R"] is not None:
        z = z + s["R"].float()
    y = z / torch.sqrt((z * z).sum(dim=1, keepdim=True) / s["c"] + EPS) * s["w"].float()
    out = _plain_eight_bits(y) if s["out"] == "i8" else (y.to(s["X"].dtype),)
    return out if s["R"] is None else out + (z.to(s["X"].dtype),)


def _plain_product(s, n):
    z = (s["X"].float() @ s["W" + n].float().t()) * (s["sx"][:, None] * s["s" + n])
    return z if s["b" + n] is None else z + s["b" + n].float()


def _plain_linear(s):
    y = _act(_plain_product(s, "w"), s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(s["out_type"])


def _plain_gated(s):
    return (_act(_plain_product(s, "g"), s["act"]) * _plain_product(s, "u")).to(s["out_type"])


def _own(s):
    from structured_rank_matmul_amd import dyra
    if s["op"] == "linear":
        return dyra.dyra_linear_quantized(s["X"], s["sx"], s["Ww"], s["sw"], bias=s["bw"], act=s["act"], residual=s["R"],
                                          out_dtype=s["out_type"])
    if s["op"] == "gated":
        return dyra.dyra_gated_quantized(s["X"], s["sx"], s["Wg"], s["sg"], s["Wu"], s["su"], bias_g=s["bg"], bias_u=s["bu"],
                                         act=s["act"], out_dtype=s["out_type"])
    if s["op"] == "quantize":
        q, scales = dyra.dyra_quantize(s["X"])
        return dyra.dyra_dequantize(q, scales, torch.bfloat16), scales
    if s["out"] == "same":
        y = dyra.dyra_norm(s["X"], s["w"], EPS, residual=s["R"])
        return y if s["R"] is not None else (y,)
    q, scales, *sums = dyra.dyra_norm_quantize(s["X"], s["w"], EPS, residual=s["R"])
    return dyra.dyra_dequantize(q, scales, torch.bfloat16), scales, *sums


def run(state):
    if own:
        return _own(state)
    if state["op"] == "quantize":
        return _plain_eight_bits(state["X"].float())
    return {"norm": _plain_norm, "linear": _plain_linear, "gated": _plain_gated}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] in ("norm", "quantize"):
        N, c, size = case["N"], case["c"], 2 if case["dtype"] == "bf16" else 4
        # rows in 8 bits are written, and read to be returned as bfloat16
        eight = case["op"] == "quantize" or case["out"] == "i8"
        out = N * c * (1 + 1 + 2) + 4 * N if eight else N * c * size
        if case["op"] == "quantize":
            return {"bytes": N * c * size + out, "flops": 3.0 * N * c}
        return {"bytes": size * (N * c * (1 + 2 * case["residual"]) + c) + out, "flops": (5.0 + 3.0 * eight) * N * c}
    N, c1, c2, size = case["N"], case["c1"], case["c2"], 2 if case["out"] == "bf16" else 4
    m = 1 if case["op"] == "linear" else 2
    return {"bytes": N * c1 + m * c1 * c2 + 4 * (N + m * c2) + size * (m * c2 * case["bias"] + N * c2 * (1 + case.get("residual", False))),
            "flops": 2.0 * m * N * c1 * c2}


# ------------------------------------------------------------------ the definitions in 64 bits

def _phi(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "quantize"):
        y, sums = s["X"].double(), []
        if case["op"] == "norm":
            if s["R"] is not None:
                y = y + s["R"].double()
                sums = [y]
            y = y * (s["w"].double() * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + EPS))
            if case["out"] == "same":
                return [y] + sums if sums else [y]
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1).clamp(min=LEAST) / 127.0
        return [torch.round(y / step[:, None]) * step[:, None], step] + sums
    x = s["X"].double()
    sums = [x.matmul(s["W" + n].double().T.contiguous()).mul_(s["sx"].double()[:, None]).mul_(s["s" + n].double()).add_(
        0.0 if s["b" + n] is None else s["b" + n].double()) for n in (("w",) if case["op"] == "linear" else ("g", "u"))]
    y = _phi(sums[0], case["act"])
    if case["op"] == "gated":
        return y * sums[1]
    return y if s["R"] is None else y + s["R"].double()
