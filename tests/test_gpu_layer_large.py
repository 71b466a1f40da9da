"""The layer norm, the codes and their products past 2^31 and 2^32 elements: rows at the
beginning, in the middle and at the end against the 64-bit forms."""

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
    torch.cuda.empty_cache()


def need(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def some(n):
    return [0, 1, n // 3, n // 2 + 1, n - 2, n - 1]


@pytest.mark.parametrize("cols", [4096, 4097])
def test_norm_rows(tg, cols):
    need(60)
    rows = 2 ** 32 // cols + 1000
    x = torch.empty(rows, cols, dtype=HALF, device="cuda").normal_()
    r = torch.empty(rows, cols, dtype=HALF, device="cuda").normal_()
    w, b = 1 + 0.1 * torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
    at = some(rows)
    want = ref.LayerNorm(x[at], r[at], weight=w, bias=b)
    y, h = tg.layer_norm(x, r, weight=w, bias=b)
    want.check(y[at], h[at], "rows")
    del y, h
    _, codes, scale = tg.layer_norm_i8(x, r, weight=w, bias=b)
    want.check_codes(codes[at], scale[at], "rows")
    del codes, scale
    codes, scale = tg.quantize_rows(x)
    exact = ref.codes_of(x[at])
    assert torch.equal(codes[at], exact[0]) and torch.equal(scale[at], exact[1])
    del codes, scale
    got = tg.layer_norm_backward(r, x, x, r, weight=w, bias=b)
    want.rows = rows
    want.check_grads((got.x[at], got.residual[at], None, None), r[at], x[at], "rows")
    # the column sums: dh is x, whose sums over rows are near those of a 64-bit pass
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    for i in range(0, rows, 65536):
        part = x[i:i + 65536].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    assert bool(((got.bias.double() - total).abs() <= 2 * ref.E * rows / 304 * size).all())


def test_codes_of_a_large_weight(tg):
    need(10)
    N, K = 2 ** 20 + 40, 4100
    b = torch.empty(N, 4112, dtype=torch.int8, device="cuda").random_(-100, 100)[:, :K]
    sb = torch.rand(N, device="cuda")
    at = some(N)
    for M in (1, 6, 12, 100):
        a = torch.randint(-100, 100, (M, K), dtype=torch.int8, device="cuda")
        sa = torch.rand(M, device="cuda")
        got = tg.gemm_i8(a, b, sa, sb, out_dtype=F32)
        want, bound = ref.i8(a, b[at], sa, sb[at])
        ref.assert_close(got[:, at], want, bound, f"{M}")


def test_a_large_result(tg):
    need(15)
    M, N, K = 70001, 65536, 96
    a = torch.randint(-100, 100, (M, K), dtype=torch.int8, device="cuda")
    b = torch.randint(-100, 100, (N, K), dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    got = tg.gemm_i8(a, b, sa, sb, out_dtype=BF16)  # (sums of 96 products pass fp16's 65504)
    at = some(M)
    want, bound = ref.i8(a[at], b, sa[at], sb)
    ref.assert_close(got[at], want, bound, "result")


def test_more_rows_than_a_slab(tg):
    """A in fp16 takes 1 GB at most at a time."""
    M, N, K = 4500, 70, 131071
    a = torch.empty(M, K, dtype=torch.int8, device="cuda").random_(-100, 100)
    b = torch.empty(N, 131072, dtype=torch.int8, device="cuda").random_(-100, 100)[:, :K]
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    bias = torch.randn(N, device="cuda")
    r = torch.randn(M, N, device="cuda")
    got = tg.gemm_i8(a, b, sa, sb, bias=bias, residual=r)
    at = some(M) + [4095, 4096, 4097]
    want, bound = ref.i8(a[at], b, sa[at], sb, bias=bias, residual=r[at])
    ref.assert_close(got[at], want, bound, "slabs")
