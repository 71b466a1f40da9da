"""tg_gemm_w4 on values that are not finite, and on weights beyond their type's range, on a
GB300: the definition's value, whatever the number of rows and the type of the result.

An infinite or NaN activation decides its products alone: a sum with it is the sum of the
row's non-finite terms a·W, an infinity times a weight of zero being NaN.  Every other row
keeps its bits.
"""

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def up(n, to):
    return -(-n // to) * to


def make(M, N, K, dtype, group, zeros, pad, scale=0.02):
    g = torch.Generator(device="cuda").manual_seed(M + 31 * N + 101 * K + group)
    groups = up(K, group) // group
    whole = torch.full((M, K + pad), NAN, device="cuda", dtype=dtype)
    whole[:, :K] = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    bq = torch.randint(0, 256, (N, up((K + 1) // 2, 16)), generator=g, device="cuda",
                       dtype=torch.uint8)[:, :(K + 1) // 2]
    s = scale * (1 + 5 * torch.rand(groups, up(N, 8), generator=g, device="cuda"))
    bzero = None
    if zeros:
        bzero = torch.randint(0, 16, (groups, up(N, 16)), generator=g, device="cuda",
                              dtype=torch.uint8)[:, :N]
    return whole[:, :K], bq, s.to(dtype)[:, :N], bzero


@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("out_dtype", [None, F32])
@pytest.mark.parametrize("dtype,group,zeros,pad", [(HALF, 64, True, 3), (BF16, 32, True, 0),
                                                   (HALF, 128, False, 8)])
@pytest.mark.parametrize("M,N,K", [(1, 80, 333), (12, 80, 333), (40, 300, 1100), (65, 300, 1100),
                                   (100, 512, 4096), (300, 5003, 1001)])
def test_infinities_and_nan(tg, M, N, K, dtype, group, zeros, pad, out_dtype, relu):
    a, bq, bscale, bzero = make(M, N, K, dtype, group, zeros, pad)
    call = lambda: tg.gemm_w4(a, bq, bscale, N, group, relu, bzero=bzero,  # noqa: E731
                              out_dtype=out_dtype)
    clean = call()
    assert bool(torch.isfinite(clean).all())
    # one infinity of either sign; two that may cancel; NaN; the last row and column too
    at = {M - 1: [(K - 1, INF)]}
    if M >= 12:
        at.update({0: [(77, -INF)], 5: [(3, INF), (200, INF)], 7: [(130, NAN)],
                   M - 2: [(64, INF), (65, -INF), (K - 2, INF)]})
    for m, terms in at.items():
        for k, v in terms:
            a[m, k] = v
    got = call()
    W = ops64.w4_weight(bq, bscale, bzero, N, K, group)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    for m, terms in at.items():
        keep[m] = False
        want = sum(v * W[:, k] for k, v in terms)
        if relu:
            want = torch.where(want > 0, want, torch.zeros_like(want))  # NaN becomes +0
        same = (got[m].double() == want) | (got[m].isnan() & want.isnan())
        assert bool(same.all()), f"row {m}: {int((~same).sum())} of {N}"
    assert torch.equal(got[keep], clean[keep])
    tg.sync_status()


@pytest.mark.parametrize("M,N,K", [(3, 80, 333), (40, 300, 1100), (65, 300, 1100), (300, 512, 4096)])
@pytest.mark.parametrize("group", [32, 128])
def test_fp32_results_of_weights_beyond_fp16(tg, M, N, K, group):
    """(code - zero)·scale up to 900 000, past fp16's 65504; every result is finite."""
    a, bq, bscale, bzero = make(M, N, K, HALF, group, True, 1, scale=10000.0)
    W = ops64.w4_weight(bq, bscale, bzero, N, K, group)
    assert float(W.abs().max()) > 65504
    c = tg.gemm_w4(a, bq, bscale, N, group, bzero=bzero, out_dtype=F32)
    want, bound = ops64.w4(a, W)
    ops64.assert_close(c, want, bound, f"{M}x{N}x{K}")
