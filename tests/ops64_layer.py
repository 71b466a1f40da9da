"""Plain 64-bit forms of the layer norm, its gradient, rows as 8-bit codes and the
products of such codes, with bounds on the error that fp32 arithmetic may leave.

Bounds.  A sum of a row's n values, each thread adding no more than n/32 of them one
after another and 16 more steps joining these, errs by at most c = (n/32 + 16)·2^-24 of
the sum of their sizes.  The differences d = v - mean(v) carry the error of the mean,
c·mean|v|, and of the sum x + r, 2^-24·(|x| + |r|); the deviation carries c of its own
and what those leave of it (at most their root mean square over the deviation).  Each
bound below is twice the sum of such terms, for the products of small errors and the
few roundings in between.
"""

from __future__ import annotations

import torch

from ops64 import U, assert_close

E = 2.0 ** -24


def mean(v):
    return v.mean(dim=1, keepdim=True)


class LayerNorm:
    def __init__(self, x, residual=None, *, weight=None, bias=None, eps=1e-5):
        self.rows, cols = x.shape
        self.c = (cols / 32 + 16) * E
        x, r = x.double(), residual.double() if residual is not None else None
        self.y = x + r if r is not None else x
        self.y_abs = x.abs() + r.abs() if r is not None else x.abs()
        self.w = weight.double() if weight is not None else torch.ones(cols, device=x.device).double()
        d = self.y - mean(self.y)
        self.s = 1.0 / torch.sqrt(mean(d * d) + eps)
        self.n = d * self.s
        self.h = self.n * self.w + (bias.double() if bias is not None else 0.0)
        d_err = E * (self.y_abs + d.abs()) + self.c * mean(self.y_abs)
        # relative, of s: its sum's own, and that of the d's
        self.s_err = self.c + 4 * E + torch.sqrt(mean(d_err * d_err)) * self.s
        self.n_err = 2 * (self.s * d_err + self.n.abs() * self.s_err)
        self.h_err = self.w.abs() * self.n_err + 4 * E * (self.n * self.w).abs()
        if bias is not None:
            self.h_err = self.h_err + 4 * E * bias.double().abs()

    def check(self, y, h, what=""):
        if y is not None:
            assert_close(y, self.y, E * self.y_abs, what + " y")
        if h is not None:
            assert_close(h, self.h, self.h_err, what + " h")

    def check_codes(self, codes, scale, what=""):
        assert codes.dtype == torch.int8 and scale.dtype == torch.float32
        most = self.h.abs().amax(dim=1)
        assert_close(scale, most / 127, 2 * self.h_err.amax(dim=1) / 127 + E * most, what + " scale")
        s = scale.double()[:, None]
        off = (codes.double() * s - self.h).abs() - (0.5 + 1e-6) * s - self.h_err
        # the largest value's code is ±127, whichever way its scale was rounded
        assert float(off.max()) <= 0, (what, float(off.max()))
        assert bool(((codes.int().abs().amax(dim=1) == 127) | (scale == 0)).all()), what

    def check_grads(self, got, dy, dh, what=""):
        zero = torch.zeros_like(self.y)
        dy = dy.double() if dy is not None else zero
        dh = dh.double() if dh is not None else zero
        dn = dh * self.w
        m2 = mean(dn * self.n)
        size = self.s * (dn.abs() + mean(dn.abs()) + self.n.abs() * mean((dn * self.n).abs()))
        dv = dy + self.s * (dn - mean(dn) - self.n * m2)
        err = 2 * ((2 * self.c + self.s_err) * size + 2 * E * dy.abs()
                   + self.s * (self.n.abs() * mean(dn.abs() * self.n_err) + self.n_err * m2.abs()))
        rows = 2 * E * self.rows
        want = (dv, dv, (dh * self.n).sum(0), dh.sum(0))
        bounds = (err, err, (dh.abs() * (self.n_err + (rows + 2 * E) * self.n.abs())).sum(0),
                  rows * dh.abs().sum(0))
        for name, g, w, b in zip(("x", "residual", "weight", "bias"), got, want, bounds):
            if g is not None:
                assert_close(g, w, b, f"{what} d{name}")


def codes_of(x):
    """(codes, scale) of quantize_rows, exactly: the scale is the fp32 number nearest to
    max|x| / 127, the codes are of the exact quotients (in 64 bits a quotient of fp32
    numbers is a half exactly when it is one)."""
    bad = ~torch.isfinite(x).all(dim=1)
    most = torch.where(bad[:, None], torch.zeros_like(x), x).double().abs().amax(dim=1)
    scale = (most / 127).float()  # (rounded once: a quotient by 127 is no tie of fp32 numbers)
    q = torch.where(scale[:, None] > 0, x.double() / scale.double()[:, None], 0.0)
    q = torch.where(bad[:, None], torch.zeros_like(q), q).round().clamp(-127, 127)
    return q.to(torch.int8), torch.where(bad, torch.full_like(scale, float("nan")), scale)


def i8(a, b, ascale, bscale, *, bias=None, relu=False, residual=None, tensor_cores=True):
    """(C, bound) of gemm_i8 in 64 bits.  The sums are whole numbers: exact in fp32 while no
    partial one passes 2^24, else each of the K/16 additions loses at most one unit of the
    24th bit.  Then two scales, the bias and the residual, each rounded once."""
    ai, bi = a.double(), b.double()
    sums, size = ai @ bi.T, ai.abs() @ bi.abs().T
    scales = ascale.double()[:, None] * bscale.double()
    v, total = sums * scales, (sums * scales).abs()
    lost = torch.where(size > 2 ** 24, size * (a.shape[1] / 16 + 2) * 2.0 ** -23, 0.0) if tensor_cores else 0.0
    bound = lost * scales.abs() + 4 * E * total
    if bias is not None:
        v = v + bias.double()
        bound = bound + 2 * E * bias.double().abs()
    if relu:
        v = torch.where(v > 0, v, torch.zeros_like(v))
    if residual is not None:
        v = v + residual.double()
        bound = bound + 2 * E * residual.double().abs()
    return v, bound


__all__ = ["LayerNorm", "codes_of", "i8", "assert_close", "U"]
