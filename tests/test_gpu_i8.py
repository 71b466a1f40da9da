"""tg_gemm_i8 against the definition on a GB300: whole sums exactly, the epilogue within
the bounds of ops64_layer.py."""

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


def make(M, N, K, *, pad=0, seed=0, low=-128, high=128):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 31 * M + 7 * N + K)

    def ints(rows, cols, ld):
        whole = torch.randint(low, high, (rows, ld), generator=g, device="cuda", dtype=torch.int8)
        return whole[:, :cols]

    a = ints(M, K, K + pad)
    b = ints(N, K, (K + 15) // 16 * 16)  # what lies behind a row is not zero
    ascale = 0.5 + torch.rand(M, generator=g, device="cuda")
    bscale = (0.5 + torch.rand(N, generator=g, device="cuda")) / 100
    return a, b, ascale, bscale, g


def check(tg, M, N, K, dtype, *, bias=False, relu=False, residual=False, pad=0, seed=0):
    a, b, sa, sb, g = make(M, N, K, pad=pad, seed=seed)
    size = 10.0 * max(K, 1) ** 0.5
    kw = dict(relu=relu, bias=size * torch.randn(N, generator=g, device="cuda") if bias else None,
              residual=(size * torch.randn(M, N, generator=g, device="cuda")).to(dtype) if residual else None)
    got = tg.gemm_i8(a, b, sa, sb, out_dtype=dtype, **kw)
    assert got.dtype == dtype and got.shape == (M, N)
    want, bound = ref.i8(a, b, sa, sb, **kw)
    ref.assert_close(got, want, bound, f"{M}x{N}x{K} {dtype} {kw.keys()}")


SIZES = [(1, 1, 1), (1, 16, 16), (1, 1000, 520), (2, 33, 65), (3, 4096, 1024), (5, 129, 4099), (7, 5003, 4099),
         (8, 640, 28672), (8, 40, 100), (9, 300, 1000), (16, 4096, 2048), (17, 257, 129), (31, 1111, 333),
         (32, 128, 128), (33, 512, 4096), (64, 3000, 1111), (65, 1024, 2000), (100, 257, 8200), (128, 640, 640),
         (200, 2048, 512), (255, 300, 300), (256, 256, 256), (257, 513, 1025), (400, 1000, 1000), (513, 129, 77),
         (1000, 2500, 640), (2100, 300, 130)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(tg, M, N, K):
    check(tg, M, N, K, F32)
    check(tg, M, N, K, HALF, bias=True, relu=True, pad=3, seed=1)
    check(tg, M, N, K, BF16, bias=True, residual=True, pad=16, seed=2)


@pytest.mark.parametrize("M", list(range(1, 20)) + [24, 40, 48, 63, 96, 160, 224, 300])
def test_rows(tg, M):
    check(tg, M, 200, 300, F32, bias=True, relu=True, residual=True)
    check(tg, M, 1024, 1024, BF16, residual=True)


@pytest.mark.parametrize("M", [1, 8, 16, 70, 300])
@pytest.mark.parametrize("N,K", [(128, 131071), (3, 20000), (20000, 3), (40000, 64), (152 * 16 + 1, 640)])
def test_long_sides(tg, M, N, K):
    check(tg, M, N, K, F32)


@pytest.mark.parametrize("M", [1, 4, 8, 20, 100, 300])
def test_sums_are_whole_numbers(tg, M):
    """Unit scales and fp32 results: the sums themselves, each exact below 2^24."""
    one = torch.ones(6000, device="cuda")
    for N, K in ((257, 1024), (1000, 333), (130, 4096)):
        a, b, _, _, _ = make(M, N, K, seed=3, low=-60, high=61)
        want = a.double() @ b.double().T
        assert float((a.double().abs() @ b.double().abs().T).max()) < 2 ** 24
        got = tg.gemm_i8(a, b, one[:M], one[:N], out_dtype=F32)
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("M", [1, 8, 40, 300])
@pytest.mark.parametrize("value", [(127, 127), (-128, -128), (-128, 127)])
def test_largest_sums(tg, M, value):
    """All products of one sign and size."""
    for K in (1024, 1041, 131071):
        a = torch.full((M, K), value[0], device="cuda", dtype=torch.int8)
        b = torch.empty(20, (K + 15) // 16 * 16, device="cuda", dtype=torch.int8)[:, :K]
        b.fill_(value[1])
        one = torch.ones(M + 20, device="cuda")
        got = tg.gemm_i8(a, b, one[:M], one[:20], out_dtype=F32)
        want, bound = ref.i8(a, b, one[:M], one[:20], tensor_cores=M > 8)
        ref.assert_close(got, want, bound, f"{M} {K} {value}")


@pytest.mark.parametrize("M", [1, 8, 30, 300])
def test_no_k(tg, M):
    a = torch.empty(M, 0, dtype=torch.int8, device="cuda")
    b = torch.empty(40, 0, dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(M, device="cuda"), torch.ones(40, device="cuda")
    bias = torch.randn(40, device="cuda")
    got = tg.gemm_i8(a, b, sa, sb, bias=bias, out_dtype=F32)
    assert torch.equal(got, bias.expand(M, 40))


def test_no_rows_or_channels(tg):
    a, b, sa, sb, _ = make(5, 40, 32)
    assert tg.gemm_i8(a[:0], b, sa[:0], sb).shape == (0, 40)
    assert tg.gemm_i8(a, b[:0], sa, sb[:0]).shape == (5, 0)


@pytest.mark.parametrize("M", [1, 7, 20, 200, 700])
def test_a_row_without_a_scale_is_nan_and_no_other(tg, M):
    a, b, sa, sb, _ = make(M, 300, 500)
    clean = tg.gemm_i8(a, b, sa, sb, out_dtype=F32)
    sa = sa.clone()
    sa[M // 2] = float("nan")
    got = tg.gemm_i8(a, b, sa, sb, out_dtype=F32)
    assert bool(got[M // 2].isnan().all())
    keep = [m for m in range(M) if m != M // 2]
    assert torch.equal(got[keep], clean[keep])
    sb = sb.clone()
    sb[7] = float("inf")
    a[0] = 0
    got = tg.gemm_i8(a, b, sa, sb, out_dtype=F32)
    assert bool(got[0, 7].isnan())  # 0 · inf
    assert bool(got[:, :7][keep].isfinite().all()) and bool(got[:, 8:][keep].isfinite().all())


@pytest.mark.parametrize("M", [1, 6, 8, 12, 64, 130, 500])
def test_results_given(tg, M):
    """Into rows of a wider matrix, in the residual's place; nothing else is written."""
    a, b, sa, sb, g = make(M, 333, 700, pad=1)
    for dtype in (HALF, F32):
        r = torch.randn(M, 333, generator=g, device="cuda").to(dtype) * 100
        want = tg.gemm_i8(a, b, sa, sb, residual=r)
        assert want.dtype == dtype
        whole = torch.full((M + 2, 340), 7.0, dtype=dtype, device="cuda")
        out = whole[1:M + 1, 3:336]
        out.copy_(r)
        got = tg.gemm_i8(a, b, sa, sb, residual=out, out=out)
        assert got is out and torch.equal(out, want)
        assert bool((whole[0] == 7).all() and (whole[-1] == 7).all() and (whole[:, :3] == 7).all()
                    and (whole[:, 336:] == 7).all())


@pytest.mark.parametrize("M", [1, 8, 50, 300])
def test_transposed_and_sliced_inputs(tg, M):
    """Any alignment of a: slices off every boundary."""
    a, b, sa, sb, _ = make(M + 1, 100, 600)
    for first in range(1, 5):
        part, weight = a[1:, first:first + 513], b[:, 16:529]
        got = tg.gemm_i8(part, weight, sa[1:], sb, out_dtype=F32)
        want, bound = ref.i8(part, weight, sa[1:], sb)
        ref.assert_close(got, want, bound, f"{first}")


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_plain_and_general_calls_agree(tg, M):
    a, b, sa, sb, g = make(M, 520, 1100)
    bias = torch.randn(520, generator=g, device="cuda")
    want = tg.gemm_i8(a, b, sa, sb, True, bias=bias)
    assert want.dtype == HALF
    assert torch.equal(tg.gemm_i8(a, b, sa, sb, True, bias=bias, out=torch.empty_like(want)), want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = tg.gemm_i8(a, b, sa, sb, True, bias=bias, stream=stream)
    stream.synchronize()
    assert torch.equal(other, want)
    # the C entry with the library's own workspace
    out = torch.empty_like(want)
    epi = tg.tg_epilogue_ex_t(1, 0, bias.data_ptr(), None, 0)
    st = tg.tg_gemm_i8(a.data_ptr(), a.stride(0), sa.data_ptr(), b.data_ptr(), b.stride(0), sb.data_ptr(),
                       out.data_ptr(), 520, M, 520, 1100, epi, None, 0,
                       torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("M,N,K", [(1, 1024, 4096), (8, 333, 5000), (24, 2000, 3000), (100, 700, 9000),
                                   (300, 256, 8192)])
def test_two_captured_graphs_at_once(tg, M, N, K):
    cases = [make(M, N, K, seed=s) for s in (1, 2)]
    want = [tg.gemm_i8(*c[:4]) for c in cases]
    graphs, got = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(tg.gemm_i8(*c[:4]))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_calls_back_to_back(tg):
    """Products of different sizes queued without a wait: each its own result."""
    cases = [make(M, N, K, seed=9) for M, N, K in ((1, 700, 900), (40, 700, 900), (8, 2000, 64), (300, 130, 5000),
                                                   (70, 4000, 256), (2, 128, 20000))]
    want = [tg.gemm_i8(*c[:4], out_dtype=F32) for c in cases]
    torch.cuda.synchronize()
    got = [[tg.gemm_i8(*c[:4], out_dtype=F32) for c in cases] for _ in range(5)]
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_refusals(tg):
    a, b, sa, sb, _ = make(4, 64, 48)
    with pytest.raises(TypeError):
        tg.gemm_i8(a.int(), b, sa, sb)
    with pytest.raises(TypeError):
        tg.gemm_i8(a, b.view(torch.uint8), sa, sb)
    with pytest.raises(ValueError):
        tg.gemm_i8(a[:, :47], b, sa, sb)
    with pytest.raises(ValueError):
        tg.gemm_i8(a, b, sa[:3], sb)
    with pytest.raises(ValueError):
        tg.gemm_i8(a, b, sa, sb.half())
    with pytest.raises(ValueError):
        tg.gemm_i8(a, b, sa, None)
    with pytest.raises(TypeError):
        tg.gemm_i8(a, b, sa, sb, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        tg.gemm_i8(a, b, sa, sb, residual=torch.zeros(4, 63, device="cuda"))
    with pytest.raises(TypeError):
        tg.gemm_i8(a, b, sa, sb, residual=torch.zeros(4, 64, device="cuda"), out_dtype=HALF)
    with pytest.raises(tg.TgemmError) as e:  # rows that do not begin on 16 bytes
        tg.gemm_i8(a[:, :40], b[:, 1:41], sa, sb)
    assert e.value.status == tg.TG_ERR_MISALIGNED
    odd = torch.zeros(64, 40, dtype=torch.int8, device="cuda")
    with pytest.raises(tg.TgemmError):
        tg.gemm_i8(a[:, :40], odd, sa, sb)


@pytest.mark.parametrize("M", [3, 100])
def test_a_wait_that_runs_out_is_reported_once(tg, M):
    """Codes that never come: the kernel gives up within its limit and returns, the status
    says so once, and the next call is right."""
    a, b, sa, sb, _ = make(M, 1000, 900)
    want = tg.gemm_i8(a, b, sa, sb)
    tg.sync_status()
    try:
        tg.tg_debug_set_wait_timeout_ns(20_000_000)
        tg.tg_debug_inject(1)
        tg.gemm_i8(a, b, sa, sb)
        with pytest.raises(tg.TgemmError) as e:
            tg.sync_status()
        assert e.value.status == tg.TG_ERR_TIMEOUT
        tg.sync_status()
    finally:
        tg.tg_debug_inject(0)
        tg.tg_debug_set_wait_timeout_ns(0)
    assert torch.equal(tg.gemm_i8(a, b, sa, sb), want)
    tg.sync_status()
