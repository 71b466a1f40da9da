"""Cases of layer norm, its gradient and 8-bit products, with their plain forms, for timing and comparison.

  norm   y = residual + x,  h = (y - mean(y)) / sqrt(var(y) + eps) ⊙ weight + bias  over each row
  grad   the gradient of ``norm`` in all of its inputs
  i8     C = out(act(ascale[m]·bscale[n]·Σ_k a[m][k]·b[n][k] + bias[n]) + R), a and b in 8-bit
         integers with a scale per row of a (token) and per row of b (channel)
  layer  a layer on activations that are not yet integers: the codes and scales of each row,
         scale = max|v| / 127 and code = v / scale to the nearest, of the layer norm of the rows or
         of the rows themselves, and the product of ``i8`` on them

A case is a dict of plain values, ``prepare`` makes its inputs on the GPU, ``run`` is one pass:
the framework's calls where ``own`` is true, elementary torch operations in 32 bits where not.
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _norm(name, op, T, D, dtype, stream, residual=True, bias=True, pad=0, empty=0, offset=0.0):
    """stream: type of the residual stream; pad: elements between the end of a row and the next
    row; empty: padding rows at the end, all zeros; offset: what all columns share."""
    return {"name": name, "op": op, "T": T, "D": D, "dtype": dtype, "stream": stream,
            "residual": residual, "bias": bias, "pad": pad, "empty": empty, "offset": offset}


def _i8(name, M, N, K, out, bias=False, relu=False, residual=False, pad=0):
    """pad: bytes between the end of a row of a and the next row."""
    return {"name": name, "op": "i8", "M": M, "N": N, "K": K, "out": out, "bias": bias,
            "relu": relu, "residual": residual, "pad": pad}


def _layer(name, M, N, K, dtype, norm, stream="", bias=True, relu=False, residual=False, pad=0):
    """norm: whether the rows go through the layer norm first; stream: as for norm."""
    return {"name": name, "op": "layer", "M": M, "N": N, "K": K, "dtype": dtype, "norm": norm,
            "stream": stream or dtype, "bias": bias, "relu": relu, "residual": residual,
            "pad": pad}


def listed():
    return [
        # one token before a block: the launch counts
        _norm("norm token 4096", "norm", 1, 4096, "bf16", "bf16"),
        # a prompt on an fp32 residual stream
        _norm("norm prompt 8192x4096", "norm", 8192, 4096, "bf16", "f32"),
        # odd width, rows off every boundary, padding rows, values far from zero
        _norm("norm odd 1021x5119", "norm", 1021, 5119, "f16", "f16", bias=False, pad=1, empty=37,
              offset=20.0),
        # a small training step, the norm alone
        _norm("grad 256x1024", "grad", 256, 1024, "f16", "f16", residual=False),
        # a training step at the MLP layer's size
        _norm("grad 8192x4096", "grad", 8192, 4096, "bf16", "bf16"),
        # odd width, fp32 stream, padding rows
        _norm("grad odd 2050x1537", "grad", 2050, 1537, "bf16", "f32", pad=5, empty=11),
        # one token through the wide projection of the MLP layer
        _i8("i8 token 28672x4096", 1, 28672, 4096, "bf16"),
        # a few tokens, no size a multiple of anything, rows off every boundary, fp32 logits
        _i8("i8 odd 7", 7, 5003, 4099, "f32", bias=True, pad=3),
        # a full decode batch on the 64-row workload's weight
        _i8("i8 batch 64 16384x8192", 64, 16384, 8192, "f16", bias=True, relu=True),
        # one token through a norm and a narrow layer: the launches count
        _layer("layer token 1024", 1, 1024, 1024, "f16", True),
        # sixteen tokens through the MLP layer's way back, added to the residual stream
        _layer("layer batch 16 4096x28672", 16, 4096, 28672, "f16", False, residual=True),
        # a prompt of 512 tokens through a norm and the wide layer
        _layer("layer prompt 512", 512, 16384, 8192, "bf16", True, stream="f32", relu=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "grad", "i8", "layer"])
    if op in ("norm", "grad"):
        D = _log(rng, 64, 16384)
        D = max(64, D // 320 * 320) if rng.random() < 0.6 else (D - 1) | 1
        T = _log(rng, 1, min(8192, 8192 * 4096 // D))
        dtype, stream = rng.choice([("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"),
                                    ("f16", "f32"), ("f32", "f32")])
        case = _norm("", op, T, D, dtype, stream, rng.random() < 0.7, rng.random() < 0.7,
                     rng.choice([0, 0, 8, 1]), T // 16 if rng.random() < 0.3 else 0,
                     rng.choice([0.0, 0.0, 5.0]))
    else:
        M = _log(rng, 1, 400) if rng.random() < 0.4 else _log(rng, 1, 64)
        N, K = _log(rng, 128, 28672), _log(rng, 128, 28672)
        while N * K > 16384 * 8192:
            N, K = _log(rng, 128, 28672), _log(rng, 128, 28672)
        if rng.random() < 0.6:
            N, K = max(128, N // 640 * 640), max(128, K // 640 * 640)
        else:
            N, K = N | 1, K | 1
        bias, relu, residual = rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.3
        pad = rng.choice([0, 0, 0, 16, 1])
        if op == "i8":
            case = _i8("", M, N, K, rng.choice(["f16", "bf16", "f32"]), bias, relu, residual, pad)
        else:
            dtype = rng.choice(["f16", "bf16"])
            case = _layer("", M, N, K, dtype, rng.random() < 0.6, rng.choice([dtype, "f32"]), bias,
                          relu, residual, pad)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _rows(rows, cols, pad, dtype, fill):
    """A rows × cols view whose rows lie cols + pad elements apart."""
    whole = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")
    view = whole[:, :cols]
    view.copy_(fill)
    return view


def _up(n, to):
    return -(-n // to) * to


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {"case": case, "eps": 1e-5}
    if case["op"] in ("norm", "grad"):
        T, D, pad = case["T"], case["D"], case["pad"]
        dtype, stream = DTYPES[case["dtype"]], DTYPES[case["stream"]]
        keep = torch.ones(T, 1, device="cuda")
        keep[T - case["empty"]:] = 0.0
        channel = torch.exp(0.5 * randn(D))  # some channels are larger than the others
        state["x"] = _rows(T, D, pad, dtype, (randn(T, D) * channel + case["offset"]) * keep)
        state["residual"] = None
        if case["residual"]:
            state["residual"] = _rows(T, D, pad, stream, 3.0 * randn(T, D) * keep)
        state["weight"] = 1.0 + 0.2 * randn(D)
        state["bias"] = 0.2 * randn(D) if case["bias"] else None
        if case["op"] == "grad":
            kind = stream if case["residual"] else dtype
            state["dy"] = _rows(T, D, pad, kind, randn(T, D) * keep)
            state["dh"] = _rows(T, D, pad, dtype, randn(T, D) * keep)
        return state

    M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
    # the weight's codes: rows of bytes, 16 bytes aligned; about normal within ±127
    codes = torch.empty(N, _up(K, 16), dtype=torch.int8, device="cuda")[:, :K]
    codes.copy_((34.0 * randn(N, K)).round_().clamp_(-127, 127))
    state["b"] = codes
    state["bscale"] = (0.5 + torch.rand(N, generator=g, device="cuda")) / (34.0 * math.sqrt(K))
    state["bias"] = randn(N) if case["bias"] else None
    out = DTYPES[case["out"] if case["op"] == "i8" else case["dtype"]]
    state["out_dtype"] = out
    state["residual"] = randn(M, N).to(out) if case["residual"] else None
    channel = torch.exp(0.8 * randn(K))
    if case["op"] == "i8":
        v = randn(M, K) * channel
        ascale = v.abs().amax(dim=1) / 127.0
        state["a"] = _rows(M, K, pad, torch.int8, (v / ascale[:, None]).round_())
        state["ascale"] = ascale
        return state
    dtype = DTYPES[case["dtype"]]
    if case["norm"]:
        state["x"] = _rows(M, K, pad, dtype, randn(M, K) * channel)
        state["stream"] = _rows(M, K, pad, DTYPES[case["stream"]], 3.0 * randn(M, K))
        state["norm_weight"] = 1.0 + 0.2 * randn(K)
        state["norm_bias"] = 0.2 * randn(K)
    else:  # what a ReLU leaves
        state["x"] = _rows(M, K, pad, dtype, (randn(M, K) * channel).clamp_(min=0))
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        import tiled_fp16_gemm_gb300 as tg
        if case["op"] == "norm":
            return tuple(tg.layer_norm(state["x"], state["residual"], weight=state["weight"],
                                       bias=state["bias"], eps=state["eps"]))
        if case["op"] == "grad":
            return tuple(tg.layer_norm_backward(state["dy"], state["dh"], state["x"],
                                                state["residual"], weight=state["weight"],
                                                bias=state["bias"], eps=state["eps"]))
        made = ()
        if case["op"] == "i8":
            a, ascale = state["a"], state["ascale"]
        elif case["norm"]:
            y, a, ascale = tg.layer_norm_i8(state["x"], state["stream"],
                                            weight=state["norm_weight"], bias=state["norm_bias"],
                                            eps=state["eps"])
            made = (y,)
        else:
            a, ascale = tg.quantize_rows(state["x"])
        c = tg.gemm_i8(a, state["b"], ascale, state["bscale"], relu=case["relu"],
                       bias=state["bias"], residual=state["residual"],
                       out_dtype=state["out_dtype"])
        return made + (c,)
    return {"norm": _plain_norm, "grad": _plain_grad, "i8": _plain_i8,
            "layer": _plain_layer}[case["op"]](state)


def _unit(v, eps):
    """Each row without its mean, over its deviation; and one over that."""
    d = v - v.mean(dim=1, keepdim=True)
    r = torch.rsqrt((d * d).mean(dim=1, keepdim=True) + eps)
    return d * r, r


def _plain_norm(s):
    x, residual = s["x"].float(), s["residual"]
    v = x + residual.float() if residual is not None else x
    h = _unit(v, s["eps"])[0] * s["weight"]
    if s["bias"] is not None:
        h = h + s["bias"]
    return v.to(residual.dtype) if residual is not None else None, h.to(s["x"].dtype)


def _plain_grad(s):
    x, residual = s["x"].float(), s["residual"]
    n, r = _unit(x + residual.float() if residual is not None else x, s["eps"])
    dh = s["dh"].float()
    dn = dh * s["weight"]
    dv = r * (dn - dn.mean(dim=1, keepdim=True) - n * (dn * n).mean(dim=1, keepdim=True))
    dv = dv + s["dy"].float()
    return (dv.to(s["x"].dtype), dv.to(residual.dtype) if residual is not None else None,
            (dh * n).sum(dim=0), dh.sum(dim=0) if s["bias"] is not None else None)


def _plain_product(s, a, ascale):
    """a: whole numbers in fp32."""
    c = (a @ s["b"].float().t()) * ascale[:, None] * s["bscale"]
    if s["bias"] is not None:
        c = c + s["bias"]
    if s["case"]["relu"]:
        c = torch.where(c > 0, c, torch.zeros_like(c))
    if s["residual"] is not None:
        c = c + s["residual"].float()
    return c.to(s["out_dtype"])


def _plain_i8(s):
    return (_plain_product(s, s["a"].float(), s["ascale"]),)


def _plain_layer(s):
    v, made = s["x"].float(), ()
    if s["case"]["norm"]:
        v = v + s["stream"].float()
        made = (v.to(s["stream"].dtype),)
        v = _unit(v, s["eps"])[0] * s["norm_weight"] + s["norm_bias"]
    scale = v.abs().amax(dim=1) / 127.0
    # in 64 bits: a quotient next to the border of two codes
    codes = torch.round(v.double() / scale.double()[:, None])
    codes = torch.where(scale[:, None] > 0, codes, torch.zeros_like(codes)).clamp(-127, 127)
    return made + (_plain_product(s, codes.float(), scale),)


# ------------------------------------------------------------------ work and exact values

def work(case):
    if case["op"] in ("norm", "grad"):
        T, D, e, r = case["T"], case["D"], SIZES[case["dtype"]], SIZES[case["stream"]]
        has, bias = int(case["residual"]), int(case["bias"])
        if case["op"] == "norm":  # read x, residual; write y, h
            return {"bytes": T * D * (2 * e + 2 * has * r) + 4 * D * (1 + bias),
                    "flops": T * D * (7 + has + bias)}
        # read x, residual, dy, dh; write dx, dresidual
        rows = 2 * e + (r if has else e) + e + 2 * has * r
        return {"bytes": T * D * rows + 4 * D * (2 + bias), "flops": T * D * (17 + has + bias)}
    M, N, K = case["M"], case["N"], case["K"]
    out = SIZES[case["out"] if case["op"] == "i8" else case["dtype"]]
    b = N * K + 4 * N + M * N * out * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
    if case["op"] == "i8":
        b += M * K + 4 * M
    else:
        b += M * K * SIZES[case["dtype"]]
        if case["norm"]:
            b += 2 * M * K * SIZES[case["stream"]] + 8 * K
    return {"bytes": b, "flops": 2 * M * N * K}


def exact(case, seed):
    """What ``run`` returns, from the definitions, in 64 bits and unrounded."""
    s = prepare(case, seed)
    if case["op"] in ("norm", "grad"):
        return _exact_norm(case, s)
    made = ()
    if case["op"] == "i8":
        a, ascale = s["a"].double(), s["ascale"].double()
    else:
        v = s["x"].double()
        if case["norm"]:
            v = v + s["stream"].double()
            made = (v,)
            v = _exact_unit(v, s["eps"]) * s["norm_weight"].double() + s["norm_bias"].double()
        # a scale is held in 32 bits, and the codes are those of the scale that is held
        ascale = (v.abs().max(dim=1).values / 127).float().double()
        a = (v / ascale.clamp(min=1e-300).unsqueeze(1)).round().clamp(-127, 127)
    c = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for n in range(0, case["N"], 4096):
        rows = s["b"][n:n + 4096].double() * s["bscale"][n:n + 4096].double().unsqueeze(1)
        c[:, n:n + 4096] = torch.mm(a, rows.t())
    c.mul_(ascale.unsqueeze(1))
    if s["bias"] is not None:
        c.add_(s["bias"].double())
    if case["relu"]:
        c.clamp_(min=0)
    if s["residual"] is not None:
        c.add_(s["residual"].double())
    return made + (c,)


def _exact_unit(v, eps):
    D = v.shape[1]
    mean = v.sum(dim=1, keepdim=True) / D
    var = (v - mean).pow(2).sum(dim=1, keepdim=True) / D
    return (v - mean) / torch.sqrt(var + eps)


def _exact_norm(case, s):
    """The values as defined; the gradients by the chain rule through torch's autograd."""
    inputs = [s[k].double() if s[k] is not None else None
              for k in ("x", "residual", "weight", "bias")]
    if case["op"] == "grad":
        inputs = [v.requires_grad_() if v is not None else v for v in inputs]
    x, residual, weight, bias = inputs
    v = x + residual if residual is not None else x
    h = _exact_unit(v, s["eps"]) * weight
    if bias is not None:
        h = h + bias
    if case["op"] == "norm":
        return v if residual is not None else None, h
    total = (v * s["dy"].double()).sum() + (h * s["dh"].double()).sum()
    asked = [t for t in inputs if t is not None]
    found = iter(torch.autograd.grad(total, asked))
    return tuple(next(found) if t is not None else None for t in inputs)
