"""tg_gemm_w4 (4-bit weights with group scales) against its 64-bit form on a GB300.

Tolerances: ops64.py (fp32 sums, one rounding of the result; above the row count
where the weights are decoded first, the rounding of each weight too).
"""

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

#: above this many rows of A the weights may have been rounded to A's type
DENSE_ROWS = 64


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def up(n, to):
    return -(-n // to) * to


def make(M, N, K, dtype, group, zeros, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + M + 31 * N + 101 * K + group)
    groups = up(K, group) // group
    a = torch.randn(M, K + pad, generator=g, device="cuda").to(dtype)[:, :K]
    # the bytes past a row's end are not zero: nothing may come of them
    bq = torch.randint(0, 256, (N, max(16, up((K + 1) // 2, 16))), generator=g, device="cuda",
                       dtype=torch.uint8)[:, :(K + 1) // 2]
    bscale = (0.02 + 0.1 * torch.rand(groups, up(N, 8), generator=g, device="cuda")).to(dtype)[:, :N]
    bzero = None
    if zeros:
        bzero = torch.randint(0, 16, (groups, up(N, 16)), generator=g, device="cuda",
                              dtype=torch.uint8)[:, :N]
    return a, bq, bscale, bzero


def check(tg, M, N, K, dtype, group, zeros, *, bias=False, relu=False, residual=False,
          out_dtype=None, pad=0, seed=0):
    a, bq, bscale, bzero = make(M, N, K, dtype, group, zeros, seed, pad)
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    r = torch.randn(M, N + pad, generator=g, device="cuda").to(dtype)[:, :N] if residual else None
    whole = torch.full((M, N + pad), 7.0, device="cuda", dtype=out_dtype or dtype)
    out = whole[:, :N]
    c = tg.gemm_w4(a, bq, bscale, N, group, relu, out, bzero=bzero, bias=b, residual=r)
    assert c is out
    W = ops64.w4_weight(bq, bscale, bzero, N, K, group)
    want, bound = ops64.w4(a, W, bias=b, relu=relu, residual=r,
                           weight_rounding=ops64.U[dtype] if M > DENSE_ROWS else 0.0)
    ops64.assert_close(c, want, bound, f"{M}x{N}x{K} {dtype} {group}")
    assert bool((whole[:, N:] == 7.0).all()), "columns past C's width were written"


HALF, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 16, 17, 31, 33, 64, 65, 200, 300])
@pytest.mark.parametrize("dtype,group,zeros", [(HALF, 128, False), (BF16, 32, True),
                                               (HALF, 64, True), (BF16, 128, False)])
def test_rows(tg, M, dtype, group, zeros):
    check(tg, M, 272, 640, dtype, group, zeros)


@pytest.mark.parametrize("N,K", [(1, 1), (1, 4096), (3, 2), (15, 31), (16, 32), (17, 33), (5, 255),
                                 (31, 256), (33, 257), (100, 511), (129, 513), (257, 1023),
                                 (64, 4099), (1000, 129), (40, 20001), (5003, 40), (2304, 2048)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_odd_sizes(tg, N, K, group):
    for M, dtype in ((1, HALF), (5, BF16), (19, HALF)):
        check(tg, M, N, K, dtype, group, True, pad=1)


@pytest.mark.parametrize("M", [1, 6, 40, 130])
@pytest.mark.parametrize("dtype", [HALF, BF16])
@pytest.mark.parametrize("bias,relu,residual,wide", [(True, False, False, False),
                                                     (False, True, False, True),
                                                     (True, True, True, False),
                                                     (True, False, True, True)])
def test_epilogue(tg, M, dtype, bias, relu, residual, wide):
    check(tg, M, 384, 768, dtype, 64, True, bias=bias, relu=relu, residual=residual,
          out_dtype=torch.float32 if wide else None, pad=3)


@pytest.mark.parametrize("M,N,K", [(1, 16384, 8192), (16, 4096, 28672), (64, 16384, 8192),
                                   (4, 28672, 4096), (2, 70000, 512)])
def test_layer_sizes(tg, M, N, K):
    check(tg, M, N, K, BF16, 128, True)


@pytest.mark.parametrize("M,N,K", [(64, 2311, 2305), (33, 5003, 3001), (17, 3001, 4099), (48, 129, 60000),
                                   (9, 9001, 4111), (16, 20000, 2048), (64, 40000, 136), (40, 4096, 1280)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_batches_of_odd_sizes(tg, M, N, K, group):
    """Row blocks shared by several blocks, ends inside units, groups and bytes."""
    check(tg, M, N, K, HALF, group, True, bias=True, pad=1)
    check(tg, M, N, K, BF16, group, False, residual=True, out_dtype=torch.float32, seed=1)


@pytest.mark.parametrize("M,N,K", [(65, 1, 1), (66, 5, 300), (100, 129, 127), (257, 600, 4099), (512, 4096, 2304),
                                   (300, 5003, 3001), (1000, 1031, 515), (70, 20000, 2048), (512, 16384, 8192),
                                   (129, 256, 60000), (3000, 2048, 1040), (70000, 64, 136)])
@pytest.mark.parametrize("dtype,group,zeros", [(HALF, 128, False), (BF16, 32, True), (HALF, 64, True)])
def test_many_rows(tg, M, N, K, dtype, group, zeros):
    """Tiles of several widths, whole and shared, with ends inside units, groups and bytes."""
    check(tg, M, N, K, dtype, group, zeros, bias=True, relu=True, residual=True, pad=1)


@pytest.mark.parametrize("M", [16, 64, 512])
@pytest.mark.parametrize("dtype,group", [(HALF, 128), (BF16, 32), (HALF, 64)])
def test_units_of_k_stay_apart(tg, M, dtype, group):
    """Row m of A picks 128 columns of W, again and again: a stage of codes, scales or zero
    points that is refilled too early, or read too late, shows in one column of results."""
    N, K = 8192, 8192
    _, bq, bscale, bzero = make(1, N, K, dtype, group, True)
    a = torch.zeros(M, K, device="cuda", dtype=dtype)
    for m in range(M):
        a[m, m % 64 * 128:m % 64 * 128 + 128] = 1
    W = ops64.w4_weight(bq, bscale, bzero, N, K, group).reshape(N, 64, 128)
    want = W.sum(2).T.repeat(-(-M // 64), 1)[:M]
    size = W.abs().sum(2).T.repeat(-(-M // 64), 1)[:M]
    bound = (K + 4) * 2.0 ** -23 * size + (ops64.U[dtype] if M > DENSE_ROWS else 0.0) * size
    for _ in range(20):
        ops64.assert_close(tg.gemm_w4(a, bq, bscale, N, group, bzero=bzero), want, bound, f"{M}")


@pytest.mark.parametrize("M", [100, 512])
def test_a_wait_that_runs_out_with_many_rows(tg, M):
    test_a_wait_that_runs_out_is_reported_once(tg, M, 4096, 4096)


@pytest.mark.parametrize("M", [65, 127, 129, 200, 400])
@pytest.mark.parametrize("dtype,group,zeros", [(HALF, 128, True), (BF16, 32, False), (BF16, 64, True)])
def test_fp32_results_round_no_weight(tg, M, dtype, group, zeros):
    """However many rows: an fp32 result has fp32 sums' error and no more."""
    N, K = 1100, 2311
    a, bq, bscale, bzero = make(M, N, K, dtype, group, zeros, 3, 1)
    r = torch.randn(M, N, device="cuda").to(dtype)
    b = torch.randn(N, device="cuda")
    c = tg.gemm_w4(a, bq, bscale, N, group, True, bzero=bzero, bias=b, residual=r,
                   out_dtype=torch.float32)
    W = ops64.w4_weight(bq, bscale, bzero, N, K, group)
    want, bound = ops64.w4(a, W, bias=b, relu=True, residual=r)
    ops64.assert_close(c, want, bound, f"{M} {dtype} {group}")


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_plain_and_general_calls_agree(tg, out_dtype):
    """A call whose result is given takes another way through the binding: the same bits."""
    a, bq, bscale, bzero = make(3, 200, 300, HALF, 64, True)
    b, r = torch.randn(200, device="cuda"), torch.randn(3, 200, device="cuda").half()
    kw = dict(relu=True, bzero=bzero, bias=b, residual=r)
    c = tg.gemm_w4(a, bq, bscale, 200, 64, out_dtype=out_dtype, **kw)
    assert c.dtype is (out_dtype or HALF) and c.shape == (3, 200)
    assert torch.equal(c, tg.gemm_w4(a, bq, bscale, 200, 64, out=torch.empty_like(c), **kw))


def test_batches_of_changing_shapes(tg):
    """One stream's workspace serves every shape: what one call leaves there does not
    show in the next."""
    for M, N, K in ((64, 2304, 2304), (64, 16384, 1024), (9, 8192, 8192), (64, 2304, 2304),
                    (33, 128, 50000), (64, 16384, 1024)):
        check(tg, M, N, K, HALF, 64, True)


@pytest.mark.parametrize("M,N,K", [(1, 2048, 2048), (8, 1000, 4096), (40, 4096, 4096)])
def test_a_wait_that_runs_out_is_reported_once(tg, M, N, K):
    """A fetch that is left out: the kernel gives up within its limit and returns, the
    status says so once, and the next call is right."""
    a, bq, bscale, bzero = make(M, N, K, HALF, 64, True)
    want = tg.gemm_w4(a, bq, bscale, N, 64, bzero=bzero)
    tg.sync_status()
    try:
        tg.tg_debug_set_wait_timeout_ns(20_000_000)
        tg.tg_debug_inject(1)
        tg.gemm_w4(a, bq, bscale, N, 64, bzero=bzero)
        with pytest.raises(tg.TgemmError) as e:
            tg.sync_status()
        assert e.value.status == tg.TG_ERR_TIMEOUT
        tg.sync_status()
    finally:
        tg.tg_debug_inject(0)
        tg.tg_debug_set_wait_timeout_ns(0)
    for _ in range(2):
        assert torch.equal(tg.gemm_w4(a, bq, bscale, N, 64, bzero=bzero), want)
    tg.sync_status()


def test_exact_on_small_integers(tg):
    """Scales of 1 and small integers: every sum is an integer below 2^24, exact in
    fp32 in any order, so the result is exact."""
    for M, N, K, group, dtype in ((1, 1024, 4096, 128, HALF), (8, 300, 1000, 32, BF16),
                                  (33, 520, 2048, 64, HALF), (100, 264, 512, 32, BF16)):
        a, bq, bscale, bzero = make(M, N, K, dtype, group, True)
        a = torch.randint(-2, 3, (M, K), device="cuda").to(dtype)
        bscale = torch.ones_like(bscale)
        full = torch.ones(bscale.shape[0], up(N, 8), device="cuda", dtype=dtype)[:, :N]
        c = tg.gemm_w4(a, bq, full, N, group, bzero=bzero, out_dtype=torch.float32)
        want = a.double() @ ops64.w4_weight(bq, full, bzero, N, K, group).T
        assert torch.equal(c.double(), want)


def test_without_zeros_is_eight(tg):
    a, bq, bscale, _ = make(3, 96, 512, HALF, 32, False)
    eight = torch.full((16, 96), 8, device="cuda", dtype=torch.uint8)
    high = eight + 16 * 5  # only the low four bits are read
    c = tg.gemm_w4(a, bq, bscale, 96, 32)
    assert torch.equal(c, tg.gemm_w4(a, bq, bscale, 96, 32, bzero=eight))
    assert torch.equal(c, tg.gemm_w4(a, bq, bscale, 96, 32, bzero=high))


@pytest.mark.parametrize("M", [1, 12])
def test_infinities_and_nan_stay_in_their_row(tg, M):
    """A row of A with an infinity: W·inf, of the sign of the weight, NaN where the
    weight is zero.  Other rows, and columns past K, know nothing of it."""
    N, K = 80, 333
    a, bq, bscale, bzero = make(M, N, K, HALF, 64, True, pad=8)
    base = torch.full((M, K + 8), float("nan"), device="cuda", dtype=HALF)
    base[:, :K] = a
    clean = tg.gemm_w4(base[:, :K], bq, bscale, N, 64, bzero=bzero)
    assert bool(torch.isfinite(clean).all())
    base[M - 1, 77] = float("inf")
    got = tg.gemm_w4(base[:, :K], bq, bscale, N, 64, bzero=bzero)
    assert torch.equal(got[:M - 1], clean[:M - 1])
    w = ops64.w4_weight(bq, bscale, bzero, N, K, 64)[:, 77]
    want = torch.where(w == 0, torch.full_like(w, float("nan")), w.sign() * float("inf"))
    assert torch.equal(got[M - 1].double().nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))


@pytest.mark.parametrize("M", [1, 5, 40, 90])
def test_residual_in_place(tg, M):
    a, bq, bscale, _ = make(M, 264, 512, BF16, 128, False)
    r = torch.randn(M, 264, device="cuda").to(BF16)
    want = tg.gemm_w4(a, bq, bscale, 264, 128, residual=r)
    got = tg.gemm_w4(a, bq, bscale, 264, 128, residual=r, out=r)
    assert got is r and torch.equal(got, want)


def test_same_bits_every_time_and_on_another_stream(tg):
    for M in (1, 16, 64, 256):
        a, bq, bscale, bzero = make(M, 1040, 4096, HALF, 64, True)
        first = tg.gemm_w4(a, bq, bscale, 1040, 64, bzero=bzero)
        for _ in range(3):
            assert torch.equal(first, tg.gemm_w4(a, bq, bscale, 1040, 64, bzero=bzero))
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        there = tg.gemm_w4(a, bq, bscale, 1040, 64, bzero=bzero, stream=other)
        torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(first, there)


@pytest.mark.parametrize("M", [1, 33, 200])
def test_in_a_graph(tg, M):
    a, bq, bscale, bzero = make(M, 512, 1024, HALF, 128, True)
    want = tg.gemm_w4(a, bq, bscale, 512, 128, bzero=bzero)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = tg.gemm_w4(a, bq, bscale, 512, 128, bzero=bzero)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tg.gemm_w4(a, bq, bscale, 512, 128, bzero=bzero, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_empty_and_k0(tg):
    _, bq, bscale, _ = make(1, 48, 64, HALF, 32, False)
    assert tg.gemm_w4(torch.empty(0, 64, device="cuda", dtype=HALF), bq, bscale, 48, 32).shape == (0, 48)
    b = torch.linspace(-1, 1, 48, device="cuda")
    a = torch.empty(3, 0, device="cuda", dtype=HALF)
    c = tg.gemm_w4(a, bq[:, :0], bscale[:0], 48, 32, True, bias=b)
    assert torch.equal(c, b.clamp(min=0).to(HALF).expand(3, 48))


def test_refusals(tg):
    a, bq, bscale, bzero = make(2, 48, 64, HALF, 32, True)
    bad = [
        (TypeError, dict(a=a.float())),
        (TypeError, dict(bq=bq.to(torch.int8))),
        (TypeError, dict(bscale=bscale.to(BF16))),
        (TypeError, dict(bzero=bzero.to(torch.int32))),
        (ValueError, dict(group=16)),
        (ValueError, dict(group=256)),
        (ValueError, dict(bq=bq[:47])),
        (ValueError, dict(bq=bq[:, :31])),
        (ValueError, dict(bscale=bscale[:1])),
        (ValueError, dict(bzero=bzero[:, :47])),
        (ValueError, dict(bq=bq.cpu())),
        (ValueError, dict(bias=torch.zeros(47, device="cuda"))),
        (TypeError, dict(residual=torch.zeros(2, 48, device="cuda"))),
        (ValueError, dict(residual=torch.zeros(2, 47, device="cuda", dtype=HALF))),
        (TypeError, dict(out_dtype=BF16)),
        (ValueError, dict(out=torch.zeros(3, 48, device="cuda", dtype=HALF))),
        (ValueError, dict(out=torch.zeros(48, 2, device="cuda", dtype=HALF).t())),
    ]
    good = dict(a=a, bq=bq, bscale=bscale, N=48, group=32, bzero=bzero)
    tg.gemm_w4(**good)
    for kind, change in bad:
        with pytest.raises(kind):
            tg.gemm_w4(**{**good, **change})
    wide = torch.zeros(48, 40, device="cuda", dtype=torch.uint8)  # rows 40 bytes apart
    with pytest.raises(tg.TgemmError) as e:
        tg.gemm_w4(a, wide[:, :32], bscale, 48, 32)
    assert e.value.status == tg.TG_ERR_MISALIGNED
    with pytest.raises(tg.TgemmError) as e:
        tg.gemm_w4(a[:1].expand(2, 64), bq, bscale, 48, 32)  # row stride 0
    assert e.value.status == tg.TG_ERR_INVALID_VALUE
