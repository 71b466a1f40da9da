"""Cases of the layer operators, with their plain forms, for timing and comparison.

The operators are the parts of a decoder block that stand around its matrix products:

  w4    C = out(act(A·Wᵀ + bias) + R), the weight in 4-bit codes with a scale (and, if wanted,
        a zero point) per group of `group` consecutive k of a row:
            W[n][k] = (code[n][k] - zero[k / group][n]) · scale[k / group][n]
  norm  y = residual + scale · gate ⊙ rms(x)·post_weight,   h = rms(y)·pre_weight:
        the norm after a block, its gate and residual scale, the residual sum and the norm
        before the next block; rms(v) = v / sqrt(mean(v²) + eps) over a row
  grad  the gradient of ``norm`` in all of its inputs

A case is a dict of plain values, ``prepare`` makes its inputs on the GPU, ``run`` is one pass:
the framework's call where ``own`` is true, elementary torch operations in 32 bits where not.
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _w4(name, M, N, K, dtype, group, zeros, bias=False, relu=False, residual=False, out="",
        pad=0):
    """pad: elements between the end of a row of A (and of C) and the next row."""
    return {"name": name, "op": "w4", "M": M, "N": N, "K": K, "dtype": dtype, "group": group,
            "zeros": zeros, "bias": bias, "relu": relu, "residual": residual,
            "out": out or dtype, "pad": pad}


def _norm(name, op, T, D, dtype, stream, post, gates, pre, pad=0, empty=0):
    """stream: type of the residual stream; gates: rows of the gate (0: no gate); empty: padding
    rows at the end, all zeros."""
    return {"name": name, "op": op, "T": T, "D": D, "dtype": dtype, "stream": stream,
            "post": post, "gates": gates, "pre": pre, "pad": pad, "empty": empty}


def listed():
    return [
        # the smallest product: one token through a narrow layer, where the launch counts
        _w4("w4 token 1024", 1, 1024, 1024, "f16", 128, False),
        # one token through the wide projection of the MLP layer, asymmetric codes
        _w4("w4 token 28672x4096", 1, 28672, 4096, "bf16", 128, True),
        # sixteen tokens through the MLP layer's way back, added to the residual stream
        _w4("w4 batch 16 4096x28672", 16, 4096, 28672, "f16", 64, True, residual=True),
        # a full decode batch on the 64-row workload's weight, the finest groups, ReLU
        _w4("w4 batch 64 16384x8192", 64, 16384, 8192, "bf16", 32, True, bias=True, relu=True),
        # a few tokens, no size a multiple of anything, rows off every boundary, fp32 logits
        _w4("w4 odd 7", 7, 5003, 4099, "f16", 32, True, bias=True, out="f32", pad=3),
        # a prompt of 512 tokens through the same weights
        _w4("w4 prompt 512", 512, 16384, 8192, "f16", 128, False, bias=True, relu=True),
        # one token between two blocks: the launch counts
        _norm("norm token 4096", "norm", 1, 4096, "bf16", "bf16", True, 1, True),
        # a prompt, fp32 residual stream, a gate per sequence of the batch
        _norm("norm prompt 8192x4096", "norm", 8192, 4096, "bf16", "f32", True, 8, True),
        # odd width, rows off every boundary, a gate per token, padding rows
        _norm("norm odd 1021x5119", "norm", 1021, 5119, "f16", "f16", True, 1021, True, pad=1,
              empty=37),
        # a small training step: plain residual sum and the next norm
        _norm("grad 256x1024", "grad", 256, 1024, "f16", "f16", False, 0, True),
        # a training step at the MLP layer's size with a learned gate per channel
        _norm("grad 8192x4096", "grad", 8192, 4096, "bf16", "bf16", True, 1, True),
        # odd width, two sequences with a gate each, fp32 stream, padding rows
        _norm("grad odd 2050x1537", "grad", 2050, 1537, "bf16", "f32", True, 2, True, pad=5,
              empty=11),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.5:
        dtype = rng.choice(["f16", "bf16"])
        M = _log(rng, 1, 400) if rng.random() < 0.4 else _log(rng, 1, 64)
        N, K = _log(rng, 256, 28672), _log(rng, 256, 28672)
        while N * K > 16384 * 8192:
            N, K = _log(rng, 256, 28672), _log(rng, 256, 28672)
        if rng.random() < 0.6:  # whole tiles and groups
            N, K = max(128, N // 640 * 640), max(128, K // 640 * 640)
        else:
            N, K = N | 1, K | 1
        case = _w4("", M, N, K, dtype, rng.choice([32, 64, 128]), rng.random() < 0.6,
                   rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.3,
                   rng.choice([dtype, dtype, "f32"]), rng.choice([0, 0, 0, 8, 1]))
    else:
        op = rng.choice(["norm", "grad"])
        D = _log(rng, 128, 16384)
        D = max(128, D // 320 * 320) if rng.random() < 0.6 else (D - 1) | 1
        T = _log(rng, 1, min(8192, 8192 * 4096 // D))
        T -= T % 5 if T > 64 else 0  # batches of 1, 2 or 5 sequences
        dtype, stream = rng.choice([("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"),
                                    ("f16", "f32"), ("f32", "f32")])
        per = rng.choice([1, 2, 5])
        gates = rng.choice([0, 1, T, per])
        if gates == per:
            T = max(per, T // per * per)
        case = _norm("", op, T, D, dtype, stream, rng.random() < 0.7, gates, rng.random() < 0.9,
                     rng.choice([0, 0, 8, 1]), T // 16 if rng.random() < 0.3 else 0)
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

    if case["op"] == "w4":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        dtype, groups = DTYPES[case["dtype"]], _up(K, group) // group
        # activations: some channels are an order larger than the others
        a = randn(M, K) * torch.exp(0.8 * randn(K))
        # codes: rows of packed nibbles, 16 bytes aligned; about normal around the middle
        nib = torch.randint(0, 256, (N, _up((K + 1) // 2, 16)), generator=g, device="cuda",
                            dtype=torch.uint8)
        scale = (0.5 + torch.rand(groups, N, generator=g, device="cuda")) / (4.6 * math.sqrt(K))
        bscale = torch.empty(groups, _up(N, 8), dtype=dtype, device="cuda")[:, :N]
        bscale.copy_(scale)
        bzero = None
        if case["zeros"]:
            bzero = torch.randint(4, 12, (groups, _up(N, 16)), generator=g, device="cuda",
                                  dtype=torch.uint8)[:, :N]
        return {"case": case, "a": _rows(M, K, case["pad"], dtype, a),
                "bq": nib[:, :(K + 1) // 2], "bscale": bscale, "bzero": bzero,
                "bias": randn(N) if case["bias"] else None,
                "residual": _rows(M, N, case["pad"], dtype, randn(M, N))
                if case["residual"] else None}

    T, D, pad = case["T"], case["D"], case["pad"]
    dtype, stream, gates = DTYPES[case["dtype"]], DTYPES[case["stream"]], case["gates"]
    keep = torch.ones(T, 1, device="cuda")
    keep[T - case["empty"]:] = 0.0
    channel = torch.exp(0.5 * randn(D))
    state = {"case": case,
             "x": _rows(T, D, pad, dtype, randn(T, D) * channel * keep),
             "residual": _rows(T, D, pad, stream, 3.0 * randn(T, D) * keep),
             "post_weight": 1.0 + 0.2 * randn(D) if case["post"] else None,
             "gate": (0.5 + 0.5 * randn(gates, D)).to(dtype) if gates else None,
             "pre_weight": 1.0 + 0.2 * randn(D) if case["pre"] else None,
             "scale": 0.7, "eps": 1e-6}
    if case["op"] == "grad":
        state["dy"] = _rows(T, D, pad, stream, randn(T, D) * keep)
        state["dh"] = _rows(T, D, pad, dtype, randn(T, D) * keep) if case["pre"] else None
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        import tiled_fp16_gemm_gb300 as tg
        if case["op"] == "w4":
            return tg.gemm_w4(state["a"], state["bq"], state["bscale"], case["N"], case["group"],
                              case["relu"], bzero=state["bzero"], bias=state["bias"],
                              residual=state["residual"], out_dtype=DTYPES[case["out"]])
        kept = {k: state[k] for k in ("post_weight", "gate", "pre_weight", "scale", "eps")}
        if case["op"] == "norm":
            return tuple(tg.norm_residual(state["x"], state["residual"], **kept))
        return tuple(tg.norm_residual_backward(state["dy"], state["dh"], state["x"],
                                               state["residual"], **kept))
    return {"w4": _plain_w4, "norm": _plain_norm, "grad": _plain_grad}[case["op"]](state)


def _plain_w4(s):
    case = s["case"]
    N, K, group = case["N"], case["K"], case["group"]
    codes = torch.stack((s["bq"] & 15, s["bq"] >> 4), dim=-1).reshape(N, -1)[:, :K].float()
    which = torch.arange(K, device="cuda") // group
    zero = s["bzero"].float()[which].t() if s["bzero"] is not None else 8.0
    weight = (codes - zero) * s["bscale"].float()[which].t()
    c = s["a"].float() @ weight.t()
    if s["bias"] is not None:
        c = c + s["bias"]
    if case["relu"]:
        c = torch.where(c > 0, c, torch.zeros_like(c))
    if s["residual"] is not None:
        c = c + s["residual"].float()
    return c.to(DTYPES[case["out"]])


def _rms(v, eps):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)


def _gate_rows(gate, T):
    """The gate's rows, one for each row of x."""
    return gate.float().repeat_interleave(T // gate.shape[0], dim=0)


def _plain_norm(s):
    x, dtype, eps = s["x"].float(), s["x"].dtype, s["eps"]
    o = x * _rms(x, eps) * s["post_weight"] if s["post_weight"] is not None else x
    if s["gate"] is not None:
        o = o * _gate_rows(s["gate"], x.shape[0])
    y = s["residual"].float() + s["scale"] * o
    h = None
    if s["pre_weight"] is not None:
        h = (y * _rms(y, eps) * s["pre_weight"]).to(dtype)
    return y.to(s["residual"].dtype), h


def _plain_grad(s):
    x, dtype, eps, scale = s["x"].float(), s["x"].dtype, s["eps"], s["scale"]
    post, pre, T = s["post_weight"], s["pre_weight"], s["x"].shape[0]
    rx = _rms(x, eps)
    m = x * rx
    o = m * post if post is not None else x
    g = _gate_rows(s["gate"], T) if s["gate"] is not None else None
    y = s["residual"].float() + scale * (o * g if g is not None else o)
    dy = s["dy"].float()
    dpre = dpost = dgate = None
    if pre is not None:
        ry = _rms(y, eps)
        n = y * ry
        dh = s["dh"].float()
        dpre = (dh * n).sum(dim=0)
        dn = dh * pre
        dy = dy + ry * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    do = scale * dy
    if g is not None:
        gates = s["gate"].shape[0]
        dgate = (do * o).reshape(gates, T // gates, -1).sum(dim=1).to(s["gate"].dtype)
        do = do * g
    dx = do
    if post is not None:
        dpost = (do * m).sum(dim=0)
        dm = do * post
        dx = rx * (dm - m * (dm * m).mean(dim=1, keepdim=True))
    return dx.to(dtype), dy.to(s["residual"].dtype), dgate, dpost, dpre


# ------------------------------------------------------------------ work and exact values

def work(case):
    if case["op"] == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        groups, e = _up(K, case["group"]) // case["group"], SIZES[case["dtype"]]
        b = N * ((K + 1) // 2) + groups * N * (e + (1 if case["zeros"] else 0)) + M * K * e
        b += M * N * SIZES[case["out"]] + (4 * N if case["bias"] else 0)
        b += M * N * e if case["residual"] else 0
        return {"bytes": b, "flops": 2 * M * N * K}
    T, D, e, r = case["T"], case["D"], SIZES[case["dtype"]], SIZES[case["stream"]]
    post, pre, gates = int(case["post"]), int(case["pre"]), case["gates"]
    if case["op"] == "norm":  # read x, residual; write y, h
        b = T * D * (e + 2 * r + pre * e) + 4 * D * (post + pre) + gates * D * e
        return {"bytes": b, "flops": T * D * (4 + 4 * post + 4 * pre)}
    # read x, residual, dy, dh; write dx, dresidual
    b = T * D * (2 * e + 3 * r + pre * e) + 8 * D * (post + pre) + 2 * gates * D * e
    return {"bytes": b, "flops": T * D * (8 + 12 * post + 12 * pre)}


def exact(case, seed):
    """What ``run`` returns, from the definitions, in 64 bits and unrounded."""
    s = prepare(case, seed)
    return _exact_w4(case, s) if case["op"] == "w4" else _exact_norm(case, s)


def _exact_w4(case, s):
    """Group by group: scale · Σ (code - zero)·a, with the sums of a apart."""
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    a = s["a"].double()
    c = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for i, k0 in enumerate(range(0, K, group)):
        k1 = min(K, k0 + group)
        part = a[:, k0:k1]
        packed = s["bq"][:, k0 // 2:(k1 + 1) // 2]
        code = torch.empty(N, 2 * packed.shape[1], dtype=torch.float64, device="cuda")
        code[:, 0::2] = packed.remainder(16)
        code[:, 1::2] = packed.div(16, rounding_mode="floor")
        zero = s["bzero"][i].double() if s["bzero"] is not None else 8.0
        c += s["bscale"][i].double() * (part @ code[:, :k1 - k0].T
                                        - zero * part.sum(dim=1, keepdim=True))
    if s["bias"] is not None:
        c += s["bias"].double()
    if case["relu"]:
        c.clamp_(min=0)
    if s["residual"] is not None:
        c += s["residual"].double()
    return c


def _exact_norm(case, s):
    """The values as defined; the gradients by the chain rule through torch's autograd."""
    x, r = s["x"].double(), s["residual"].double()
    post, pre, gate = (s[k].double() if s[k] is not None else None
                       for k in ("post_weight", "pre_weight", "gate"))
    inputs = [v.requires_grad_() if v is not None and case["op"] == "grad" else v
              for v in (x, r, gate, post, pre)]

    def unit(v):
        return v / torch.sqrt(v.pow(2).sum(dim=1, keepdim=True) / case["D"] + s["eps"])

    branch = unit(x) * post if post is not None else x
    if gate is not None:
        gates = case["gates"]
        branch = (branch.reshape(gates, -1, case["D"]) * gate[:, None, :]).reshape(x.shape)
    y = r + s["scale"] * branch
    h = unit(y) * pre if pre is not None else None
    if case["op"] == "norm":
        return y, h
    total = (y * s["dy"].double()).sum()
    if h is not None:
        total = total + (h * s["dh"].double()).sum()
    asked = [v for v in inputs if v is not None]
    found = iter(torch.autograd.grad(total, asked))
    return tuple(next(found) if v is not None else None for v in inputs)
