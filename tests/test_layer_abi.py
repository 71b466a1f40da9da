"""Argument checks of the layer norm, the codes and their products through the C ABI
(each before any CUDA call: no GPU is needed) and through Python."""

import ctypes

import pytest

OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
F16, BF16, F32 = 0, 1, 2
NULL = None


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    t.library()
    return t


def has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


def norm(tg, **change):
    base = dict(dtype=BF16, stream_dtype=F32, rows=6, cols=40, x=256, ldx=40, residual=256, ldr=40,
                weight=256, bias=256, eps=1e-5)
    return tg.tg_layer_norm_t(**{**base, **change})


SHARED = [
    (dict(dtype=5), INVALID),
    (dict(stream_dtype=F16), INVALID),
    (dict(dtype=F32, stream_dtype=BF16), INVALID),
    (dict(rows=-1), INVALID),
    (dict(rows=2 ** 31), INVALID),
    (dict(cols=-1), INVALID),
    (dict(cols=131072, ldx=200000, ldr=200000), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(x=NULL), INVALID),
    (dict(ldx=39), INVALID),
    (dict(ldr=39), INVALID),
    (dict(x=257), MISALIGNED),
    (dict(residual=258), MISALIGNED),
    (dict(weight=258), MISALIGNED),
    (dict(bias=258), MISALIGNED),
]


@pytest.mark.parametrize("change,want", SHARED)
def test_norm_arguments(tg, change, want):
    n = norm(tg, **change)
    wide = 200000
    assert tg.tg_layer_norm(n, 4096, wide, 4096, wide, None) == want
    assert tg.tg_layer_norm_i8(n, 4096, wide, 4096, wide, 4096, None) == want
    assert tg.tg_layer_norm_backward(n, tg.tg_layer_norm_grad_t(), None) == want


def test_norm_results(tg):
    n = norm(tg)
    call = lambda *a: tg.tg_layer_norm(n, *a, None)  # noqa: E731
    assert call(4096, 39, 4096, 40) == INVALID
    assert call(4096, 40, 4096, 39) == INVALID
    assert call(4098, 40, 4096, 40) == MISALIGNED
    assert call(4096, 40, 4097, 40) == MISALIGNED
    assert call(None, 0, None, 0) == INVALID  # no output
    bare = norm(tg, residual=None)
    assert tg.tg_layer_norm(bare, 4096, 40, 4096, 40, None) == INVALID  # y without residual
    for empty in (norm(tg, rows=0), norm(tg, cols=0, ldx=0, ldr=0)):
        assert tg.tg_layer_norm(empty, 4096, 40, 4096, 40, None) == OK
        assert tg.tg_layer_norm_i8(empty, None, 0, 4096, 40, 4096, None) == OK
    assert tg.library().tg_layer_norm(None, 256, 40, 256, 40, None) == INVALID
    codes = lambda *a: tg.tg_layer_norm_i8(n, *a, None)  # noqa: E731
    assert codes(None, 0, 4097, 39, 4096) == INVALID
    assert codes(None, 0, None, 40, 4096) == INVALID
    assert codes(None, 0, 4097, 40, None) == INVALID
    assert codes(None, 0, 4097, 40, 4098) == MISALIGNED
    assert codes(4098, 40, 4097, 40, 4096) == MISALIGNED


@pytest.mark.parametrize("change,want", [
    (dict(dtype=3), INVALID), (dict(x=NULL), INVALID), (dict(codes=NULL), INVALID),
    (dict(scale=NULL), INVALID), (dict(ldx=39), INVALID), (dict(ldc=39), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=131072, ldx=131072, ldc=131072), INVALID),
    (dict(x=257), MISALIGNED), (dict(scale=258), MISALIGNED),
    (dict(rows=0), OK), (dict(cols=0), OK),
])
def test_quantize_arguments(tg, change, want):
    args = dict(dtype=F16, x=256, ldx=40, codes=257, ldc=40, scale=256, rows=6, cols=40)
    assert tg.tg_quantize_rows(**{**args, **change}, stream=None) == want


@pytest.mark.parametrize("norm_change,grad,want", [
    ({}, dict(dy=4098, lddy=40), MISALIGNED),
    ({}, dict(dy=4096, lddy=39), INVALID),
    ({}, dict(dh=4097, lddh=40), MISALIGNED),
    ({}, dict(dx=4096, lddx=39), INVALID),
    ({}, dict(dresidual=4098, lddr=40), MISALIGNED),
    ({}, dict(dweight=4098), MISALIGNED),
    ({}, dict(dbias=4098), MISALIGNED),
    ({}, dict(workspace=4104, workspace_bytes=1 << 30), MISALIGNED),
    ({}, dict(workspace=4096, workspace_bytes=6 * 40 * 8 - 1), INVALID),
    (dict(residual=None), dict(dresidual=4096, lddr=40), INVALID),
    (dict(weight=None), dict(dweight=4096), INVALID),
    (dict(cols=0), {}, OK),
])
def test_gradient_arguments(tg, norm_change, grad, want):
    g = tg.tg_layer_norm_grad_t(**grad)
    assert tg.tg_layer_norm_backward(norm(tg, **norm_change), g, None) == want


def test_gradient_without_its_struct(tg):
    n = norm(tg)
    assert tg.library().tg_layer_norm_backward(ctypes.byref(n), None, None) == INVALID


def test_workspaces(tg):
    assert tg.tg_layer_norm_backward_workspace(6, 40) == 6 * 40 * 8
    assert tg.tg_layer_norm_backward_workspace(0, 40) == 0
    for sizes in ((-1, 4), (4, -1), (2 ** 31, 4), (4, 131072)):
        assert tg.tg_layer_norm_backward_workspace(*sizes) == -1
    for sizes in ((-1, 4, 4), (4, 2 ** 31, 4), (4, 4, 131072)):
        assert tg.tg_gemm_i8_workspace(*sizes) == -1
    assert tg.tg_gemm_i8_workspace(0, 4, 4) >= 0 and tg.tg_gemm_i8_workspace(1, 40, 40) >= 0


I8 = dict(A=257, lda=72, Ascale=256, B=256, ldb=80, Bscale=256, C=256, ldc=40, M=20, N=40, K=72,
          epi=None, workspace=None, workspace_bytes=0)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), INVALID),
    (dict(N=2 ** 31), INVALID),
    (dict(K=-5), INVALID),
    (dict(K=131072, lda=131072, ldb=131072), INVALID),
    (dict(A=NULL), INVALID),
    (dict(Ascale=NULL), INVALID),
    (dict(B=NULL), INVALID),
    (dict(Bscale=NULL), INVALID),
    (dict(C=NULL), INVALID),
    (dict(lda=71), INVALID),
    (dict(ldb=64), INVALID),
    (dict(ldc=39), INVALID),
    (dict(workspace=256, workspace_bytes=-1), INVALID),
    (dict(ldb=88), MISALIGNED),
    (dict(B=264), MISALIGNED),
    (dict(Ascale=258), MISALIGNED),
    (dict(Bscale=258), MISALIGNED),
    (dict(C=257), MISALIGNED),
    (dict(workspace=264, workspace_bytes=1 << 40), MISALIGNED),
    (dict(M=0), OK),
    (dict(N=0), OK),
    (dict(M=0, A=NULL, Ascale=NULL, C=NULL, lda=0), OK),
])
def test_i8_arguments(tg, change, want):
    assert tg.tg_gemm_i8(**{**I8, **change}, stream=None) == want


@pytest.mark.parametrize("epi,want", [
    ((2, F16, None, None, 0), INVALID),
    ((0, 3, None, None, 0), INVALID),
    ((0, F16, None, 256, 39), INVALID),
    ((0, F16, 258, None, 0), MISALIGNED),
    ((0, F16, None, 257, 40), MISALIGNED),
    ((0, F32, None, 258, 40), MISALIGNED),
])
def test_i8_epilogue_arguments(tg, epi, want):
    e = tg.tg_epilogue_ex_t(*epi)
    assert tg.tg_gemm_i8(**{**I8, "epi": e}, stream=None) == want
    wide = tg.tg_epilogue_ex_t(0, F32, None, None, 0)
    assert tg.tg_gemm_i8(**{**I8, "C": 258, "epi": wide}, stream=None) == MISALIGNED


@pytest.mark.skipif(has_gpu(), reason="a device is present")
def test_valid_calls_without_a_device(tg):
    assert tg.tg_gemm_i8(**I8, stream=None) == UNSUPPORTED
    assert tg.tg_gemm_i8(**{**I8, "K": 0, "A": NULL, "B": NULL}, stream=None) == UNSUPPORTED
    assert tg.tg_layer_norm(norm(tg), 4096, 40, 4096, 40, None) == UNSUPPORTED
    assert tg.tg_layer_norm_i8(norm(tg), None, 0, 4097, 40, 4096, None) == UNSUPPORTED
    assert tg.tg_quantize_rows(F16, 256, 40, 257, 40, 256, 6, 40, None) == UNSUPPORTED
    assert tg.tg_layer_norm_backward(norm(tg), tg.tg_layer_norm_grad_t(), None) == UNSUPPORTED


def test_python_refusals(tg):
    """Tensors that are not on a GPU, or not tensors."""
    torch = pytest.importorskip("torch")
    if torch.version.cuda is None:
        pytest.skip("needs PyTorch with CUDA")
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        tg.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.layer_norm_i8(x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.quantize_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.layer_norm_backward(None, x, x)
    with pytest.raises(TypeError):
        tg.layer_norm([1.0])
    with pytest.raises(ValueError, match="2-D"):
        tg.quantize_rows(torch.zeros(16))
    with pytest.raises(TypeError, match="float16"):
        tg.quantize_rows(torch.zeros(2, 16, dtype=torch.int32))
    codes, scale = torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gemm_i8(codes, codes, scale, scale)
    with pytest.raises(TypeError):
        tg.gemm_i8(None, codes, scale, scale)
