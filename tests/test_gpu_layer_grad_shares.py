"""The layer norm's gradient at the numbers of rows at which an SM has two: in two blocks, and past the
shares that the second launch takes at once in two groups of a block."""

import pytest

import ops64_layer as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    yield t
    t.sync_status()


@pytest.mark.parametrize("dtype,stream,pad", [(BF16, BF16, 0), (HALF, F32, 8), (F32, F32, 0), (BF16, BF16, 1)])
@pytest.mark.parametrize("cols", [72, 512, 1023, 1032, 1536, 2048, 2567, 4096])
def test_two_rows_of_an_sm(tg, dtype, stream, pad, cols):
    for rows in (152, 153, 200, 255, 256, 257, 300, 304, 305):
        g = torch.Generator(device="cuda").manual_seed(rows + cols)

        def mat(kind):
            return torch.randn(rows, cols + pad, generator=g, device="cuda").to(kind)[:, :cols]

        x, r, dy, dh = mat(dtype), mat(stream), mat(stream), mat(dtype)
        kw = dict(residual=r, weight=1 + 0.3 * torch.randn(cols, generator=g, device="cuda"),
                  bias=torch.randn(cols, generator=g, device="cuda"))
        got = tg.layer_norm_backward(dy, dh, x, **kw)
        ref.LayerNorm(x, **kw).check_grads(got, dy, dh, f"{rows}x{cols}")
        again = tg.layer_norm_backward(dy, dh, x, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
