"""The block norms' gradient where the residual stream is not finite, on a GB300."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("dtype,stream", [(BF16, F32), (HALF, HALF)])
@pytest.mark.parametrize("cols,pad", [(96, 0), (1001, 1), (4096, 0), (9000, 0), (9001, 3), (32768, 0)])
def test_gradient_without_dh_does_not_read_y(tg, cols, pad, dtype, stream, pre):
    """Without dh nothing depends on y = residual + ..., so a residual with infinities and
    NaN gives the bits of a finite one: dresidual = dy, and the others from dy alone."""
    rows = 37
    g = torch.Generator(device="cuda").manual_seed(cols + pad)
    mat = lambda t: torch.randn(rows, cols + pad, generator=g, device="cuda").to(t)[:, :cols]  # noqa: E731
    vec = lambda: 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")  # noqa: E731
    x, r, dy = mat(dtype), mat(stream), mat(stream)
    kept = dict(post_weight=vec(), gate=mat(dtype)[:1], scale=0.7, pre_weight=vec() if pre else None)
    want = tg.norm_residual_backward(dy, None, x, r, **kept)
    r[3, 5], r[9, cols - 1], r[20, 0] = float("inf"), float("-inf"), float("nan")
    got = tg.norm_residual_backward(dy, None, x, r, **kept)
    tg.sync_status()
    assert torch.equal(got.residual, dy)
    for name, a, b in zip(got._fields, got, want):
        assert (a is None) == (b is None)
        assert a is None or torch.equal(a, b), name
