"""Calls as the first CUDA work of a host thread, on a GB300: no context is current there
before the library's own calls."""

import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def in_new_thread(f):
    got = []

    def run():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("M", [1, 12, 40, 100, 600])
def test_4bit_products(tg, M):
    N, K = 5000, 1024
    a = torch.randn(M, K, device="cuda").half()
    bq = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    scale = torch.full((K // 64, N), 0.01, device="cuda", dtype=torch.half)
    for out_dtype in (None, torch.float32):
        want = tg.gemm_w4(a, bq, scale, N, 64, out_dtype=out_dtype)
        out = torch.zeros_like(want)
        call = lambda: tg.gemm_w4(a, bq, scale, N, 64, out=out)  # noqa: E731, B023
        assert torch.equal(in_new_thread(call), want)


def test_dense_products(tg):
    for M, N, K in ((16, 512, 1024), (600, 520, 776), (2048, 2048, 1024)):
        a, b = torch.randn(M, K, device="cuda").half(), torch.randn(K, N, device="cuda").half()
        want = tg.gemm(a, b)
        # tensor maps of other addresses than the first call's
        a2, b2, out = a.clone(), b.clone(), torch.empty_like(want)
        assert torch.equal(in_new_thread(lambda: tg.gemm(a2, b2, out=out)), want)  # noqa: B023


def test_norms(tg):
    x, r, d = (torch.randn(64, 512, device="cuda") for _ in range(3))
    w = torch.rand(512, device="cuda")
    want = (*tg.norm_residual(x, r, pre_weight=w), *tg.norm_residual_backward(d, d, x, r, pre_weight=w))
    y, h = torch.empty_like(x), torch.empty_like(x)
    got = in_new_thread(lambda: (*tg.norm_residual(x, r, pre_weight=w, out=y, normed=h),
                                 *tg.norm_residual_backward(d, d, x, r, pre_weight=w)))
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
