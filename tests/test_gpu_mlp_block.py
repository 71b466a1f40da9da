"""examples/mlp_block.py: the 4-bit products and the block norms as they are used
together, each stage against its 64-bit form on a GB300."""

import importlib.util
import os

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def check_product(a, w, c, K, relu):
    W = ops64.w4_weight(w["bq"], w["bscale"], w["bzero"], w["N"], K, w["group"])
    want, bound = ops64.w4(a, W, relu=relu)
    ops64.assert_close(c, want, bound, f"{tuple(a.shape)} {w['N']}")


@pytest.mark.parametrize("dtype,group", [(torch.bfloat16, 128), (torch.float16, 32)])
@pytest.mark.parametrize("rows", [1, 33])
def test_stages(ex, dtype, group, rows):
    dim, hidden = 264, 1033
    stack = ex.Stack(2, dim, hidden, group=group, dtype=dtype)
    x = torch.randn(rows, dim, device="cuda").to(dtype)
    _, h = ex.tg.norm_residual(x, pre_weight=stack.first)
    for i, norm in enumerate(stack.norms):
        f = ex.tg.gemm_w4(h, relu=True, **stack.up[i])
        check_product(h, stack.up[i], f, dim, True)
        o = ex.tg.gemm_w4(f, **stack.down[i])
        check_product(f, stack.down[i], o, hidden, False)
        y, h = ex.tg.norm_residual(o, x, scale=stack.scale, **norm)
        ops64.Norm(o, x, scale=stack.scale, **norm).check(y, h, f"block {i}")
        x = y


def test_quantised_weights_are_near(ex):
    """Half a step of the group, and half a step more from the rounded zero point."""
    w = torch.randn(50, 200, device="cuda")
    q = ex.quantise(w, 32, torch.float16)
    W = ops64.w4_weight(q["bq"], q["bscale"], q["bzero"], 50, 200, 32)
    g = torch.arange(200, device="cuda") // 32
    step = q["bscale"].double()[g].T
    assert bool(((W - w.double()).abs() <= 1.02 * step).all())


def test_a_token_as_a_graph(ex):
    """Every replay gives the bits of the calls made one by one."""
    stack = ex.Stack(2, 512, 2048)
    token = ex.Token(stack)
    for seed in range(3):
        x = torch.randn(1, 512, device="cuda").to(stack.dtype) * (seed + 1)
        h = token.step(x).clone()
        assert torch.equal(h, stack.run(x)[1])
    ex.tg.sync_status()


def test_tuning_lowers_the_loss(ex):
    stack = ex.Stack(2, 256, 512)
    x = torch.randn(100, 256, device="cuda").to(stack.dtype)
    target = 1.5 * stack.run(x)[1].float()
    losses = [ex.tune(stack, x, target, 0.2) for _ in range(4)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
