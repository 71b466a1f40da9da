"""Plain 64-bit forms of the operators beside the GEMM, with bounds on the error
that fp32 arithmetic may leave, for the tests of the CUDA kernels.

Bounds.  u = 2^-p is the unit roundoff of a type (p = 11, 8, 24 bits for fp16,
bf16, fp32): storing v errs by at most u·|v|, and by 2^-25 where fp16 is
subnormal.  A value summed from K fp32 products errs by at most
K·2^-23·Σ|terms| (each step by one unit in the last place of the running sum at
most, as a tensor core that truncates may; a rounding addition errs by half).
"""

from __future__ import annotations

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}


def assert_close(got, want, bound, what=""):
    """|got - want| <= u·|want| + bound for every element; want in 64 bits."""
    assert tuple(got.shape) == tuple(want.shape), (what, got.shape, want.shape)
    g = got.double()
    tol = U[got.dtype] * want.abs() + TINY[got.dtype] + bound
    bad = ~((g - want).abs() <= tol)
    if bool(bad.any()):
        i = int(((g - want).abs() - tol).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; "
                             f"worst {g.flatten()[i]} against {want.flatten()[i]} "
                             f"(bound {tol.expand_as(want).flatten()[i]})")


# ------------------------------------------------------------------ 4-bit weights

def w4_weight(bq, bscale, bzero, N, K, group):
    """W in 64 bits from codes, scales and zero points."""
    b = bq[:N].to(torch.int64)
    code = torch.stack((b % 16, b // 16), dim=2).reshape(N, -1)[:, :K].double()
    g = torch.arange(K, device=bq.device) // group
    zero = (bzero[:, :N].to(torch.int64) % 16).double()[g].T if bzero is not None else 8.0
    return (code - zero) * bscale[:, :N].double()[g].T


def w4(a, weight, *, bias=None, relu=False, residual=None, weight_rounding=0.0):
    """(C, bound): C = act(a·Wᵀ + bias) + R in 64 bits; ``weight_rounding`` is the
    u of the type that each weight was rounded to, 0 where none was."""
    a = a.double()
    K = a.shape[1]
    c = a @ weight.T
    size = a.abs() @ weight.abs().T
    # K products, one more multiplication by the scale per group, bias, residual
    total = size.clone()
    if bias is not None:
        c = c + bias.double()
        total = total + bias.double().abs()
    if relu:
        c = torch.where(c > 0, c, torch.zeros_like(c))
    if residual is not None:
        c = c + residual.double()
        total = total + residual.double().abs()
    return c, (K + 4) * 2.0 ** -23 * total + weight_rounding * size


# ------------------------------------------------------------------ norms

def _gate_rows(gate, rows):
    return gate.double().reshape(-1, gate.shape[-1]).repeat_interleave(
        rows // (gate.shape[0] if gate.dim() == 2 else 1), dim=0)


class Norm:
    """Values of the norms around a block in 64 bits, row by row, with majorants
    (the same sums over absolute values) that scale the bounds."""

    def __init__(self, x, residual=None, *, post_weight=None, gate=None, scale=1.0,
                 pre_weight=None, eps=1e-6):
        rows, cols = x.shape
        self.rows, self.cols, self.scale, self.eps = rows, cols, scale, eps
        self.x = x.double()
        self.post = post_weight.double() if post_weight is not None else None
        self.pre = pre_weight.double() if pre_weight is not None else None
        self.gate_shape = gate.shape if gate is not None else None
        self.g = _gate_rows(gate, rows) if gate is not None else None
        self.rx = 1.0 / torch.sqrt((self.x ** 2).mean(dim=1, keepdim=True) + eps)
        self.m = self.x * self.rx
        self.o = self.m * self.post if self.post is not None else self.x
        branch = self.o * self.g if self.g is not None else self.o
        r = residual.double() if residual is not None else torch.zeros_like(self.x)
        self.y = r + scale * branch
        self.y_abs = r.abs() + abs(scale) * branch.abs()
        self.ry = 1.0 / torch.sqrt((self.y ** 2).mean(dim=1, keepdim=True) + eps)
        self.n = self.y * self.ry
        self.n_abs = self.y_abs * self.ry
        self.h = self.n * self.pre if self.pre is not None else None
        self.h_abs = self.n_abs * self.pre.abs() if self.pre is not None else None
        # relative error of a row's statistics: no thread adds more than cols / 32
        # squares one after another, 16 more steps join them and finish
        self.c = (cols / 32 + 16) * 2.0 ** -24
        # cancellation in y magnifies the error of its sum of squares
        self.k = 1.0 + 2.0 * (self.y_abs ** 2).sum(dim=1, keepdim=True) / (
            (self.y ** 2).sum(dim=1, keepdim=True) + eps * cols)

    def check(self, y, h, what=""):
        if y is not None:
            assert_close(y, self.y, 2 * self.c * self.y_abs, what + " y")
        if h is not None:
            assert_close(h, self.h, 4 * self.c * self.k * self.h_abs, what + " h")

    def grads(self, dy, dh):
        """(dx, dresidual, dgate, dpost, dpre) and their bounds."""
        mean = lambda v: v.mean(dim=1, keepdim=True)  # noqa: E731
        sum_gates = lambda v: v.reshape(  # noqa: E731
            self.gate_shape[0] if len(self.gate_shape) == 2 else 1, -1, self.cols
        ).sum(dim=1).reshape(self.gate_shape)
        zero = torch.zeros_like(self.x)
        d = dy.double() if dy is not None else zero
        d_abs = d.abs()
        dpre = dpre_b = dpost = dpost_b = dgate = dgate_b = None
        # every product and mean below errs by at most 8 c of its majorant, times
        # the row's cancellation factor; a sum over rows adds a unit per row
        c = 8 * self.c * self.k
        over_rows = 2.0 ** -23 * self.rows
        if self.pre is not None:
            dh = dh.double() if dh is not None else zero
            dpre, dpre_b = (dh * self.n).sum(0), ((c + over_rows) * dh.abs() * self.n_abs).sum(0)
            dn = dh * self.pre
            d = d + self.ry * (dn - self.n * mean(dn * self.n))
            d_abs = d_abs + self.ry * (dn.abs() + self.n_abs * mean(dn.abs() * self.n_abs))
        dr, dr_b = d, c * d_abs
        d, d_abs = self.scale * d, abs(self.scale) * d_abs
        if self.g is not None:
            dgate = sum_gates(d * self.o)
            dgate_b = sum_gates((c + over_rows) * d_abs * self.o.abs())
            d, d_abs = d * self.g, d_abs * self.g.abs()
        if self.post is not None:
            dpost = (d * self.m).sum(0)
            dpost_b = ((c + over_rows) * d_abs * self.m.abs()).sum(0)
            dm, dm_abs = d * self.post, d_abs * self.post.abs()
            d = self.rx * (dm - self.m * mean(dm * self.m))
            d_abs = self.rx * (dm_abs + self.m.abs() * mean(dm_abs * self.m.abs()))
        return (d, dr, dgate, dpost, dpre), (2 * c * d_abs, dr_b, dgate_b, dpost_b, dpre_b)

    def check_grads(self, got, dy, dh, what=""):
        want, bounds = self.grads(dy, dh)
        for name, g, w, b in zip(("x", "residual", "gate", "post", "pre"), got, want, bounds):
            if g is not None:
                assert_close(g, w, b, f"{what} d{name}")
