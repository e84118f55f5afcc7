"""Cases of the feed-forward operators: the linear layer with its epilogue, the
gated pair of products, the router and the mixture-of-experts layer for a few
tokens.

A case names its operator in "op" and holds plain sizes and choices.  With
``own`` false, ``run`` computes the operator by elementary torch operations in
float32, rounded once at the end; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BF16_FLOPS_MOST = 3.8e12   # a drawn case costs no more than the largest listed one
F32_FLOPS_MOST = 2.0e11
EXPERT_BYTES_MOST = 2.8e9

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


# ------------------------------------------------------------------ cases

def linear(name, N, c1, c2, dtype="bf16", act="none", bias=False, residual=False, out="same", pad=0):
    """pad: elements between the rows of X (X a column slice of a wider matrix)."""
    return {"name": name, "op": "linear", "N": N, "c1": c1, "c2": c2, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "out": out, "pad": pad}


def gated(name, N, c1, c2, dtype="bf16", act="silu", bias=False, pad=0):
    return {"name": name, "op": "gated", "N": N, "c1": c1, "c2": c2, "dtype": dtype, "act": act, "bias": bias,
            "pad": pad}


def route(name, T, E, k, dtype="f32", score="softmax", renormalise=True, masked=False):
    """masked: some experts of some rows at -inf, some rows with nothing left."""
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score,
            "renormalise": renormalise, "masked": masked}


def moe(name, T, E, k, c, f, dtype="bf16", act="silu", residual=True, dropped=False):
    """dropped: some of the chosen experts' places are empty (-1)."""
    return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "c": c, "f": f, "dtype": dtype, "act": act,
            "residual": residual, "dropped": dropped}


def listed():
    return [
        # ViT-L block, 128 images x 201 tokens: fc1 with its bias and GELU, fc2 with its bias and the residual stream
        linear("vitl fc1 gelu", 25728, 1024, 4096, act="gelu", bias=True),
        linear("vitl fc2 residual", 25728, 4096, 1024, bias=True, residual=True),
        # the float32 layer of one instance of 256 tokens, the smallest product
        linear("linear384 f32", 256, 384, 384, dtype="f32", act="gelu", bias=True, residual=True),
        # one token through an attention block's output projection, added to the residual stream
        linear("one token", 1, 4096, 4096, residual=True),
        # a head of an odd number of classes over one clip's frames and one more, X a slice of a wider matrix, float32 out
        linear("odd head", 1501, 1280, 1003, bias=True, out="f32", pad=24),
        # the gate and up products of a Llama-style MLP: 8 prompts of 2048 tokens, and 16 sequences decoding
        gated("gated prefill", 16384, 4096, 14336),
        gated("gated decode", 16, 4096, 14336),
        # routers: a decoding batch, and a prefill with masked experts and rows with none left
        route("route decode", 16, 64, 8),
        route("route prefill", 16384, 128, 8, masked=True),
        # expert layers: one token through small experts, a decoding batch over many, one over a few wide ones
        moe("moe one token", 1, 64, 8, 2048, 1024),
        moe("moe batch", 48, 64, 6, 2048, 1408, dropped=True),
        moe("moe wide", 16, 8, 2, 4096, 14336),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _tokens(rng, flops_per_token, dtype, most):
    fit = int((BF16_FLOPS_MOST if dtype == "bf16" else F32_FLOPS_MOST) / flops_per_token)
    return _between(rng, 1, max(1, min(most, fit)))


def draw(rng):
    op = rng.choice(("linear", "gated", "route", "moe"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "linear":
        c1, c2 = 8 * _between(rng, 4, 1792), _between(rng, 1, 16384)
        if rng.random() < 0.5:
            c2 = -(-c2 // 32) * 32
        case = linear("", _tokens(rng, 2.0 * c1 * c2, dtype, 32768), c1, c2, dtype=dtype, act=rng.choice(ACTS),
                      bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                      out="f32" if rng.random() < 0.3 else "same", pad=rng.choice((0, 0, 0, 8, 200)))
    elif op == "gated":
        c1, c2 = 8 * _between(rng, 4, 1024), _between(rng, 1, 14336)
        if rng.random() < 0.5:
            c2 = -(-c2 // 32) * 32
        case = gated("", _tokens(rng, 4.0 * c1 * c2, dtype, 32768), c1, c2, dtype=dtype, act=rng.choice(ACTS),
                     bias=rng.random() < 0.5, pad=rng.choice((0, 0, 0, 8, 200)))
    elif op == "route":
        E = _between(rng, 2, 512)
        case = route("", _between(rng, 1, 32768), E, _between(rng, 1, min(E, 16)), dtype=dtype,
                     score=rng.choice(("softmax", "softmax", "sigmoid")), renormalise=rng.random() < 0.6,
                     masked=rng.random() < 0.5)
    else:
        E = _between(rng, 4, 128)
        c = 8 * _between(rng, 32, 640)
        size = 2 if dtype == "bf16" else 4
        f_most = max(64, min(14336, int(EXPERT_BYTES_MOST / (3 * E * c * size))))
        case = moe("", _between(rng, 1, 64), E, _between(rng, 1, min(E, 8)), c, 8 * _between(rng, 8, f_most // 8),
                   dtype=dtype, act=rng.choice(("silu", "silu", "gelu", "relu")), residual=rng.random() < 0.5,
                   dropped=rng.random() < 0.4)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _rows(n, c, gen, dtype, pad=0):
    """Rows of unit RMS with a few large channels, as after a norm; pad > 0: a column slice of a wider matrix."""
    x = torch.randn(n, c + pad, generator=gen, device=DEVICE)
    x[:, :: max(1, c // 6)] *= 8.0
    x = x / x.square().mean(dim=1, keepdim=True).sqrt()
    return x.to(dtype)[:, pad // 2 // 8 * 8:][:, :c]


def _weight(shape, gen, dtype):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=dtype).mul_(shape[-1] ** -0.5)


def _choices(T, E, k, gen):
    """k distinct experts a token, and weights that sum to one."""
    ids = torch.rand(T, E, generator=gen, device=DEVICE).argsort(dim=1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand(T, k, generator=gen, device=DEVICE) + 0.1
    return ids, w / w.sum(dim=1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    t = TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("linear", "gated"):
        N, c1, c2 = case["N"], case["c1"], case["c2"]
        s["X"] = _rows(N, c1, gen, t, case["pad"])
        if case["op"] == "linear":
            s["out_type"] = torch.float32 if case["out"] == "f32" else t
            s["W"] = _weight((c2, c1), gen, t)
            s["b"] = torch.randn(c2, generator=gen, device=DEVICE).to(t) if case["bias"] else None
            s["R"] = (2.0 * torch.randn(N, c2, generator=gen, device=DEVICE)).to(s["out_type"]) if case["residual"] else None
        else:
            s["Wg"], s["Wu"] = _weight((c2, c1), gen, t), _weight((c2, c1), gen, t)
            s["bg"] = torch.randn(c2, generator=gen, device=DEVICE).to(t) if case["bias"] else None
            s["bu"] = torch.randn(c2, generator=gen, device=DEVICE).to(t) if case["bias"] else None
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = 2.0 * torch.randn(T, E, generator=gen, device=DEVICE)
        if case["masked"]:
            logits[torch.rand(T, E, generator=gen, device=DEVICE) < 0.3] = -math.inf
            logits[torch.rand(T, generator=gen, device=DEVICE) < 0.05] = -math.inf
        s["logits"] = logits.to(t)
    else:
        T, E, k, c, f = (case[n] for n in ("T", "E", "k", "c", "f"))
        s["X"] = _rows(T, c, gen, t)
        s["Wg"], s["Wu"], s["Wd"] = _weight((E, f, c), gen, t), _weight((E, f, c), gen, t), _weight((E, c, f), gen, t)
        s["ids"], s["w"] = _choices(T, E, k, gen)
        if case["dropped"]:
            s["ids"][torch.rand(T, k, generator=gen, device=DEVICE) < 0.2] = -1
        s["R"] = (0.5 * torch.randn(T, c, generator=gen, device=DEVICE)).to(t) if case["residual"] else None
    return s


# ------------------------------------------------------------------ one pass

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _product(x, w, b):
    z = x.float() @ w.float().t()
    return z if b is None else z + b.float()


def _plain_linear(s):
    y = _act(_product(s["X"], s["W"], s["b"]), s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(s["out_type"])


def _plain_gated(s):
    h = _act(_product(s["X"], s["Wg"], s["bg"]), s["act"]) * _product(s["X"], s["Wu"], s["bu"])
    return h.to(s["X"].dtype)


def _plain_route(s):
    logits = s["logits"].float()
    top, at = torch.sort(logits, dim=1, descending=True, stable=True)
    top, at = top[:, :s["k"]], at[:, :s["k"]]
    none = top == -math.inf
    if s["score"] == "softmax":
        m = logits.amax(dim=1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        total = torch.exp(logits - m).sum(dim=1, keepdim=True)
        w = torch.exp(top - m) / torch.where(total == 0, torch.ones_like(total), total)
    else:
        w = 1.0 / (1.0 + torch.exp(-top))
    if s["renormalise"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return torch.where(none, torch.full_like(at, -1), at).to(torch.int32), torch.where(none, torch.zeros_like(w), w)


def _plain_moe(s):
    """Every expert for every token, weighted by what the token gives it (0 for most)."""
    x = s["X"].float()
    h = _act(torch.matmul(x, s["Wg"].float().transpose(1, 2)), s["act"]) * torch.matmul(x, s["Wu"].float().transpose(1, 2))
    o = torch.matmul(h, s["Wd"].float().transpose(1, 2))
    experts = torch.arange(s["E"], device=x.device, dtype=torch.int32)
    given = ((s["ids"][:, :, None] == experts) * s["w"][:, :, None]).sum(dim=1)
    y = (given.t()[:, :, None] * o).sum(dim=0)
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(s["X"].dtype)


def _own(s):
    from structured_rank_matmul_amd import dyra
    if s["op"] == "linear":
        return dyra.dyra_linear(s["X"], s["W"], bias=s["b"], act=s["act"], residual=s["R"], out_dtype=s["out_type"])
    if s["op"] == "gated":
        return dyra.dyra_gated(s["X"], s["Wg"], s["Wu"], bias_g=s["bg"], bias_u=s["bu"], act=s["act"])
    if s["op"] == "route":
        return dyra.dyra_route(s["logits"], s["k"], score=s["score"], renormalise=s["renormalise"])
    return dyra.dyra_moe(s["X"], s["Wg"], s["Wu"], s["Wd"], s["ids"], s["w"], act=s["act"], residual=s["R"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "gated": _plain_gated, "route": _plain_route, "moe": _plain_moe}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        N, c1, c2 = case["N"], case["c1"], case["c2"]
        out = 4 if case["out"] == "f32" else size
        return {"bytes": size * (N * c1 + c1 * c2 + c2 * case["bias"]) + out * N * c2 * (1 + case["residual"]),
                "flops": 2.0 * N * c1 * c2}
    if case["op"] == "gated":
        N, c1, c2 = case["N"], case["c1"], case["c2"]
        return {"bytes": size * (N * c1 + 2 * c1 * c2 + N * c2 + 2 * c2 * case["bias"]), "flops": 4.0 * N * c1 * c2}
    if case["op"] == "route":
        return {"bytes": size * case["T"] * case["E"] + 8 * case["T"] * case["k"],
                "flops": 4.0 * case["T"] * case["E"]}
    T, E, k, c, f = (case[n] for n in ("T", "E", "k", "c", "f"))
    kept = k * (0.8 if case["dropped"] else 1.0)
    experts = E * (1.0 - (1.0 - kept / E) ** T)   # distinct ones, for evenly spread choices
    return {"bytes": size * (3 * experts * c * f + T * c * (2 + case["residual"])) + 8 * T * k,
            "flops": 6.0 * T * kept * c * f}


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
    if case["op"] == "linear":
        y = s["X"].double().matmul(s["W"].double().T.contiguous())
        if s["b"] is not None:
            y += s["b"].double()
        y = _phi(y, case["act"])
        return y if s["R"] is None else y + s["R"].double()
    if case["op"] == "gated":
        x = s["X"].double()
        g, u = (x.matmul(s[w].double().T.contiguous()) + (s[b].double() if s[b] is not None else 0.0)
                for w, b in (("Wg", "bg"), ("Wu", "bu")))
        return _phi(g, case["act"]) * u
    if case["op"] == "route":
        k, l = case["k"], s["logits"].double().cpu().numpy()
        ids = torch.from_numpy((-l).argsort(axis=1, kind="stable")[:, :k].copy())
        l = torch.from_numpy(l)
        top = l.gather(1, ids)
        w = torch.softmax(l, dim=1).gather(1, ids) if case["score"] == "softmax" else torch.sigmoid(top)
        w = torch.nan_to_num(w, nan=0.0)           # rows with every expert masked
        gone = torch.isneginf(top)
        w[gone] = 0.0
        ids[gone] = -1
        if case["renormalise"]:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
        return ids.to(torch.int32), w
    x, ids, w = s["X"].double(), s["ids"].cpu(), s["w"].double()
    y = torch.zeros_like(x) if s["R"] is None else s["R"].double()
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        t, j = t.to(x.device), j.to(x.device)
        g, u, d = (s[n][e].double() for n in ("Wg", "Wu", "Wd"))
        h = _phi(x[t].matmul(g.T.contiguous()), case["act"]) * x[t].matmul(u.T.contiguous())
        y.index_add_(0, t, w[t, j][:, None] * h.matmul(d.T.contiguous()))
    return y
