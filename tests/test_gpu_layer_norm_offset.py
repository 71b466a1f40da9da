"""A mean far from zero costs the layer norm no digits: its results against 64 bits, with a bound that
does not grow with the mean.

All kernels take the differences from a value near the mean first.  What is left of the mean's size is the rounding of the
sum x + residual, 2^-24 of it, and none where there is no residual.  Everything else is of the size of
the differences d: their own rounding, and their sums, in which a value passes through 64 additions
at most (32 of a thread's pairs, 1 of the pair, 5 of a warp, and those of the warps' and blocks' sums), and
in rows of more than 32768 columns through cols / 256 + 10 (of 256 threads, and a block's sum).  As everywhere, twice the sum of such terms.
"""

import pytest

import ops64_layer as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


class Shifted(ref.LayerNorm):
    def __init__(self, x, residual=None, *, weight=None, bias=None, eps=1e-5):
        super().__init__(x, residual, weight=weight, bias=bias, eps=eps)
        cols = x.shape[1]
        self.c = (64 if cols <= 32768 else cols / 256 + 10) * ref.E
        d = (self.y - ref.mean(self.y)).abs()
        d_err = 2 * ref.E * d + self.c * ref.mean(d)
        if residual is not None:
            d_err = d_err + ref.E * self.y.abs() + ref.E * ref.mean(self.y.abs())
        self.s_err = self.c + 4 * ref.E + torch.sqrt(ref.mean(d_err * d_err)) * self.s
        self.n_err = 2 * (self.s * d_err + self.n.abs() * self.s_err)
        self.h_err = self.w.abs() * self.n_err + 4 * ref.E * (self.n * self.w).abs()
        if bias is not None:
            self.h_err = self.h_err + 4 * ref.E * bias.double().abs()


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    yield t
    t.sync_status()


def case(rows, cols, dtype, stream, offset, pad):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)

    def mat(kind, size=1.0, off=0.0):
        return (size * torch.randn(rows, cols + pad, generator=g, device="cuda") + off).to(kind)[:, :cols]

    x, r = mat(dtype, 2.0, offset), mat(stream, 3.0, offset / 3) if stream is not None else None
    kw = dict(weight=1 + 0.3 * torch.randn(cols, generator=g, device="cuda"),
              bias=0.3 * torch.randn(cols, generator=g, device="cuda"))
    return x, r, mat(stream or dtype), mat(dtype), kw


# (fp16 and bf16 hold no such deviations beside a large mean: smaller offsets)
KINDS = [(F32, None, -3000.0), (F32, F32, 500.0), (F32, None, 1e5), (HALF, None, 100.0), (BF16, F32, 40.0),
         (HALF, HALF, -60.0)]


@pytest.mark.parametrize("dtype,stream,offset", KINDS)
@pytest.mark.parametrize("cols,pad", [(40, 0), (256, 0), (1000, 0), (1023, 1), (2560, 0), (4096, 0), (5119, 0),
                                      (9001, 1), (12808, 0), (16384, 0), (16391, 0), (32768, 0), (32769, 0), (131071, 0)])
def test_rows(tg, dtype, stream, offset, cols, pad):
    for rows in (3, 300 if cols < 100000 else 30):
        x, r, dy, dh, kw = case(rows, cols, dtype, stream, offset, pad)
        want = Shifted(x, r, **kw)
        y, h = tg.layer_norm(x, r, **kw)
        want.check(y, h, f"{rows}x{cols}")
        _, codes, scale = tg.layer_norm_i8(x, r, **kw)
        want.check_codes(codes, scale, f"{rows}x{cols}")


@pytest.mark.parametrize("dtype,stream,offset", KINDS)
@pytest.mark.parametrize("cols,pad", [(40, 0), (1000, 0), (1023, 1), (4096, 0), (9001, 1), (16384, 0), (40000, 0), (70001, 0),
                                      (131071, 0)])
def test_gradients(tg, dtype, stream, offset, cols, pad):
    """Rows in one block, on the blocks of a cluster, and read again for each pass."""
    for rows in (3, 200 if cols < 70000 else 40):
        x, r, dy, dh, kw = case(rows, cols, dtype, stream, offset, pad)
        got = tg.layer_norm_backward(dy, dh, x, r, **kw)
        Shifted(x, r, **kw).check_grads(got, dy, dh, f"{rows}x{cols}")
