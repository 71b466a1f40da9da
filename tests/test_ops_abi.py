"""Argument checks of the operators beside the GEMM (tg_gemm_w4, tg_norm_residual,
tg_norm_residual_backward) through the C ABI: each is made before any CUDA call,
so no GPU is needed.  The last check of a valid call is the device."""

import ctypes

import pytest

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
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


W4 = dict(in_dtype=F16, A=256, Bq=256, Bscale=256, Bzero=256, C=256, M=2, N=40, K=72, group=32,
          lda=72, ldbq=48, ldbs=40, ldbz=48, ldc=40)


@pytest.mark.parametrize("change,want", [
    (dict(in_dtype=F32), INVALID),
    (dict(in_dtype=7), INVALID),
    (dict(group=0), INVALID),
    (dict(group=48), INVALID),
    (dict(group=256), INVALID),
    (dict(M=-1), INVALID),
    (dict(N=2 ** 31), INVALID),
    (dict(K=-5), INVALID),
    (dict(A=NULL), INVALID),
    (dict(Bq=NULL), INVALID),
    (dict(Bscale=NULL), INVALID),
    (dict(C=NULL), INVALID),
    (dict(lda=71), INVALID),
    (dict(ldbq=32), INVALID),
    (dict(ldbs=39), INVALID),
    (dict(ldbz=39), INVALID),
    (dict(ldc=39), INVALID),
    (dict(A=257), MISALIGNED),
    (dict(C=257), MISALIGNED),
    (dict(Bq=264), MISALIGNED),
    (dict(Bscale=264), MISALIGNED),
    (dict(Bzero=264), MISALIGNED),
    (dict(ldbq=40), MISALIGNED),
    (dict(ldbs=44), MISALIGNED),
    (dict(ldbz=40), MISALIGNED),
    (dict(M=0), 0),
    (dict(N=0), 0),
    (dict(M=0, A=NULL, C=NULL, lda=0), 0),
])
def test_w4_arguments(tg, change, want):
    assert tg.tg_gemm_w4(**{**W4, **change}, epi=None, stream=None) == want


@pytest.mark.parametrize("epi,want", [
    ((2, F16, None, None, 0), INVALID),
    ((0, BF16, None, None, 0), INVALID),
    ((0, F16, None, 256, 39), INVALID),
    ((0, F16, 258, None, 0), MISALIGNED),
    ((0, F16, None, 257, 40), MISALIGNED),
])
def test_w4_epilogue_arguments(tg, epi, want):
    e = tg.tg_epilogue_ex_t(*epi)
    assert tg.tg_gemm_w4(**W4, epi=e, stream=None) == want
    wide = tg.tg_epilogue_ex_t(0, F32, None, None, 0)
    assert tg.tg_gemm_w4(**{**W4, "C": 258}, epi=wide, stream=None) == MISALIGNED


def norm(tg, **change):
    base = dict(dtype=BF16, stream_dtype=F32, rows=6, cols=40, x=256, ldx=40, residual=256, ldr=40,
                post_weight=256, gate=256, ldg=40, gate_rows=2, pre_weight=256, scale=1.0, eps=1e-6)
    return tg.tg_norm_t(**{**base, **change})


SHARED = [
    (dict(dtype=5), INVALID),
    (dict(stream_dtype=F16), INVALID),
    (dict(dtype=F32, stream_dtype=BF16), INVALID),
    (dict(rows=-1), INVALID),
    (dict(rows=2 ** 31), INVALID),
    (dict(cols=-1), INVALID),
    (dict(cols=32769, ldx=40000, ldr=40000, ldg=40000), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(x=NULL), INVALID),
    (dict(ldx=39), INVALID),
    (dict(ldr=39), INVALID),
    (dict(ldg=39), INVALID),
    (dict(gate_rows=0), INVALID),
    (dict(gate_rows=4), INVALID),
    (dict(gate_rows=12), INVALID),
    (dict(x=257), MISALIGNED),
    (dict(residual=258), MISALIGNED),
    (dict(gate=257), MISALIGNED),
    (dict(post_weight=258), MISALIGNED),
    (dict(pre_weight=258), MISALIGNED),
]


@pytest.mark.parametrize("change,want", SHARED)
def test_norm_arguments(tg, change, want):
    n = norm(tg, **change)
    assert tg.tg_norm_residual(n, 4096, 40, 4096, 40, None) == want
    assert tg.tg_norm_residual_backward(n, tg.tg_norm_grad_t(), None) == want


def test_norm_results(tg):
    n = norm(tg)
    call = lambda *a: tg.tg_norm_residual(n, *a, None)  # noqa: E731
    assert call(4096, 39, 4096, 40) == INVALID
    assert call(4096, 40, 4096, 39) == INVALID
    assert call(4098, 40, 4096, 40) == MISALIGNED
    assert call(4096, 40, 4097, 40) == MISALIGNED
    assert call(4096, 40, None, 0) == INVALID  # pre_weight without h
    bare = norm(tg, pre_weight=None)
    assert tg.tg_norm_residual(bare, 4096, 40, 4096, 40, None) == INVALID
    assert tg.tg_norm_residual(bare, None, 0, None, 0, None) == 0
    for empty in (norm(tg, rows=0), norm(tg, cols=0, ldx=0, ldr=0, ldg=0)):
        assert tg.tg_norm_residual(empty, 4096, 40, 4096, 40, None) == 0
    lib = tg.library()
    assert lib.tg_norm_residual(None, 256, 40, 256, 40, None) == INVALID


@pytest.mark.parametrize("norm_change,grad,want", [
    ({}, dict(dy=4098, lddy=40), MISALIGNED),
    ({}, dict(dy=4096, lddy=39), INVALID),
    ({}, dict(dh=4097, lddh=40), MISALIGNED),
    ({}, dict(dx=4096, lddx=39), INVALID),
    ({}, dict(dresidual=4098, lddr=40), MISALIGNED),
    ({}, dict(dgate=4096, lddg=39), INVALID),
    ({}, dict(dpost_weight=4098), MISALIGNED),
    ({}, dict(dpre_weight=4098), MISALIGNED),
    (dict(pre_weight=None), dict(dh=4096, lddh=40), INVALID),
    (dict(pre_weight=None), dict(dpre_weight=4096), INVALID),
    (dict(post_weight=None), dict(dpost_weight=4096), INVALID),
    (dict(gate=None), dict(dgate=4096, lddg=40), INVALID),
    (dict(cols=0), {}, 0),
])
def test_gradient_arguments(tg, norm_change, grad, want):
    g = tg.tg_norm_grad_t(**grad)
    assert tg.tg_norm_residual_backward(norm(tg, **norm_change), g, None) == want


def test_gradient_without_its_struct(tg):
    n = norm(tg)
    assert tg.library().tg_norm_residual_backward(ctypes.byref(n), None, None) == INVALID


@pytest.mark.skipif(has_gpu(), reason="a device is present")
def test_valid_calls_without_a_device(tg):
    assert tg.tg_gemm_w4(**W4, epi=None, stream=None) == UNSUPPORTED
    assert tg.tg_gemm_w4(**{**W4, "K": 0}, epi=None, stream=None) == UNSUPPORTED
    assert tg.tg_norm_residual(norm(tg), 4096, 40, 4096, 40, None) == UNSUPPORTED
    assert tg.tg_norm_residual_backward(norm(tg), tg.tg_norm_grad_t(), None) == UNSUPPORTED
