"""Layer norm and 8-bit products on a GB300 at the sizes where their launches divide the work in
different ways: few and many rows, warps with all of their columns or not, tiles that clusters share
in equal parts or in even runs."""

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


def norm_case(rows, cols, dtype, stream, pad=0):
    g = torch.Generator(device="cuda").manual_seed(131 * rows + cols)

    def mat(kind, factor=1.0):
        return (factor * torch.randn(rows, cols + pad, generator=g, device="cuda")).to(kind)[:, :cols]

    kept = dict(residual=mat(stream, 3.0), weight=1 + 0.3 * torch.randn(cols, generator=g, device="cuda"),
                bias=0.3 * torch.randn(cols, generator=g, device="cuda"))
    return mat(dtype, 2.0), kept, mat(stream), mat(dtype)


@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (HALF, F32)])
@pytest.mark.parametrize("cols", [256, 512, 768, 1536, 2560, 3584, 5120, 12808, 16384, 16391])
def test_norm(tg, dtype, stream, cols):
    """Rows around those that 152 SMs hold at a time, with 512 threads each and with more."""
    for rows in (1, 40, 151, 153, 430, 440, 700, 1300):
        if rows * cols > 8000000:
            continue
        x, kept, _, _ = norm_case(rows, cols, dtype, stream)
        want = ref.LayerNorm(x, **kept)
        y, h = tg.layer_norm(x, **kept)
        want.check(y, h, f"{rows}x{cols}")
        y2, codes, scale = tg.layer_norm_i8(x, **kept)
        assert torch.equal(y, y2)
        want.check_codes(codes, scale, f"{rows}x{cols}")
        got, size = tg.quantize_rows(h)
        codes, scale = ref.codes_of(h)
        assert torch.equal(got, codes) and torch.equal(size, scale)


@pytest.mark.parametrize("dtype,stream,pad", [(BF16, BF16, 0), (HALF, F32, 0), (BF16, F32, 1)])
@pytest.mark.parametrize("cols", [40, 640, 1024, 1030, 4096, 9728, 9736, 16384])
def test_gradient(tg, dtype, stream, pad, cols):
    """Rows around one and two of an SM, and several groups in a block."""
    for rows in (1, 2, 152, 153, 160, 161, 256, 257, 305, 1000):
        if rows * cols > 6000000:
            continue
        x, kept, dy, dh = norm_case(rows, cols, dtype, stream, pad)
        want = ref.LayerNorm(x, **kept)
        want.check_grads(tg.layer_norm_backward(dy, dh, x, **kept), dy, dh, f"{rows}x{cols}")


@pytest.mark.parametrize("rows,cols", [(100, 640), (200, 1024), (1000, 1000), (300, 12000)])
def test_one_column_sum_without_the_other(tg, rows, cols):
    x, kept, dy, dh = norm_case(rows, cols, BF16, BF16)
    both = tg.layer_norm_backward(dy, dh, x, **kept)
    weight = tg.layer_norm_backward(dy, dh, x, kept["residual"], weight=kept["weight"])
    bias = tg.layer_norm_backward(dy, dh, x, kept["residual"], bias=kept["bias"])
    assert weight.bias is None and torch.equal(weight.weight, both.weight)
    assert bias.weight is None and torch.equal(bias.bias, both.bias)


def codes_case(M, N, K, low=-128, high=128, seed=0):
    g = torch.Generator(device="cuda").manual_seed(7919 * M + 31 * N + K + seed)

    def ints(rows):
        return torch.randint(low, high, (rows, (K + 15) // 16 * 16), generator=g, device="cuda",
                             dtype=torch.int8)[:, :K]

    return ints(M), ints(N), 0.5 + torch.rand(M, generator=g, device="cuda"), \
        (0.5 + torch.rand(N, generator=g, device="cuda")) / 100, g


# rows of a; weights: one tile in up to 64 parts, a few tiles, as many as clusters, more
SHARED = [(m, n, k) for m in (33, 64, 100, 300)
          for n, k in ((100, 8200), (1024, 8192), (2100, 4096), (9700, 2048), (12000, 4100), (19500, 640))]


@pytest.mark.parametrize("M,N,K", SHARED)
def test_products(tg, M, N, K):
    a, b, sa, sb, g = codes_case(M, N, K)
    bias = 100 * torch.randn(N, generator=g, device="cuda")
    residual = (100 * torch.randn(M, N, generator=g, device="cuda")).to(BF16)
    got = tg.gemm_i8(a, b, sa, sb, True, bias=bias, residual=residual)
    want, bound = ref.i8(a, b, sa, sb, bias=bias, relu=True, residual=residual)
    ref.assert_close(got, want, bound, f"{M}x{N}x{K}")
    assert torch.equal(got, tg.gemm_i8(a, b, sa, sb, True, bias=bias, residual=residual))


@pytest.mark.parametrize("M,N,K", [(17, 9700, 4096), (50, 300, 4096), (64, 4096, 4096), (130, 1000, 4000),
                                   (300, 2000, 3999)])
def test_shared_sums_are_exact(tg, M, N, K):
    """Unit scales: sums below 2^24, in whatever parts they are taken."""
    a, b, _, _, _ = codes_case(M, N, K, -60, 61)
    one = torch.ones(max(M, N), device="cuda")
    assert K * 60 * 60 < 2 ** 24
    got = tg.gemm_i8(a, b, one[:M], one[:N], out_dtype=F32)
    assert torch.equal(got.double(), a.double() @ b.double().T)


@pytest.mark.parametrize("M", [40, 64, 260])
@pytest.mark.parametrize("value", [127, -128])
def test_the_largest_sums_of_shared_tiles(tg, M, value):
    """K = 131071 products of (-128)² = 2^14: whole sums 2^31 - 2^14, a multiple of 2^14 in every
    part, so exact in fp32; those of 127² lose one unit of the 24th bit per addition at most."""
    K, N = 131071, 300
    a = torch.full((M, K), value, device="cuda", dtype=torch.int8)
    b = torch.empty(N, K + 1, device="cuda", dtype=torch.int8)[:, :K]
    b.fill_(value)
    one = torch.ones(N, device="cuda")
    got = tg.gemm_i8(a, b, one[:M], one, out_dtype=F32).double()
    want = float(K * value * value)
    assert bool((got == want).all() if value == -128 else ((got - want).abs() <= want * K / 16 * 2.0 ** -23).all())
    assert bool((got > 0).all())


@pytest.mark.parametrize("M,N,K", [(64, 1024, 8192), (40, 9700, 2048), (300, 300, 4096), (200, 19500, 640)])
def test_a_workspace_with_anything_in_it(tg, M, N, K):
    """What a workspace holds before the call is no part of its result; nothing past it is written."""
    a, b, sa, sb, _ = codes_case(M, N, K)
    want = tg.gemm_i8(a, b, sa, sb)
    size = tg.tg_gemm_i8_workspace(M, N, K)
    work = torch.full((size + 4096,), 0x7f, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    for _ in range(3):
        work[:size] = 0x7f
        out.zero_()
        st = tg.tg_gemm_i8(a.data_ptr(), a.stride(0), sa.data_ptr(), b.data_ptr(), b.stride(0), sb.data_ptr(),
                           out.data_ptr(), N, M, N, K, None, work.data_ptr(), size,
                           torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(out, want)
        assert bool((work[size:] == 0x7f).all())


def test_captured_products_that_share_tiles(tg):
    """Two graphs, each with two products, replayed at once on two streams."""
    cases = [codes_case(64, 1024, 8192, seed=s) + codes_case(100, 2100, 4096, seed=s) for s in (1, 2)]

    def run(c):
        return tg.gemm_i8(*c[:4], out_dtype=F32), tg.gemm_i8(*c[5:9], out_dtype=F32)

    want = [run(c) for c in cases]
    graphs, got = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(c))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))


@pytest.mark.parametrize("M,N,K", [(64, 1024, 8192), (40, 9700, 2048)])
def test_a_wait_that_runs_out_in_a_shared_tile(tg, M, N, K):
    """One cluster of a tile gives up: reported once, the others end, and the next call is right."""
    a, b, sa, sb, _ = codes_case(M, N, K)
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
