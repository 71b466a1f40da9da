"""The 4-bit products and the block norms where offsets pass 32 bits, and 4-bit weights whose
scales are subnormal, on a GB300."""

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    yield t
    torch.cuda.empty_cache()


def need(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


#: rows that are looked at: the first, those around offsets of 2^31 and 2^32 elements, the last
def some_rows(rows, cols):
    at = {0, 1, rows - 2, rows - 1}
    for edge in (2 ** 31 // cols, 2 ** 32 // cols):
        at |= {r for r in range(edge - 1, edge + 2) if r < rows}
    return torch.tensor(sorted(at), device="cuda")


def random_rows(rows, cols, dtype, seed):
    """A matrix of one random block of rows, again and again, each time scaled otherwise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(rows, cols, device="cuda", dtype=dtype)
    block = torch.randn(4096, cols, generator=g, device="cuda", dtype=F32)
    for i, r in enumerate(range(0, rows, 4096)):
        n = min(4096, rows - r)
        out[r:r + n] = block[:n] * (1 + i % 7 / 8)
    return out


@pytest.mark.parametrize("rows,cols,gates", [(524289, 8200, 1), (262145, 16392, 262145)])
def test_norms(tg, rows, cols, gates):
    need(90)
    x, r = (random_rows(rows, cols, BF16, s) for s in (1, 2))
    kept = dict(post_weight=1 + 0.1 * torch.rand(cols, device="cuda"), scale=0.6,
                gate=random_rows(gates, cols, BF16, 3), pre_weight=1 + 0.1 * torch.rand(cols, device="cuda"))
    at = some_rows(rows, cols)
    part = dict(kept, gate=kept["gate"][at] if gates > 1 else kept["gate"])
    ref = ops64.Norm(x[at], r[at], eps=1e-6, **part)
    y, h = tg.norm_residual(x, r, **kept)
    ref.check(y[at], h[at], f"{rows}x{cols}")
    del y, h
    dy, dh = (random_rows(rows, cols, BF16, s) for s in (4, 5))
    grads = tg.norm_residual_backward(dy, dh, x, r, **kept)
    want, bounds = ref.grads(dy[at], dh[at])
    ops64.assert_close(grads.x[at], want[0], bounds[0], "dx")
    ops64.assert_close(grads.residual[at], want[1], bounds[1], "dresidual")
    if gates > 1:
        ops64.assert_close(grads.gate[at], want[2], bounds[2], "dgate")


@pytest.mark.parametrize("M,N,K,group", [(140001, 32768, 128, 32), (70, 65544, 131072, 128),
                                         (2500, 65544, 65600, 64), (3, 65544, 131072, 128),
                                         (33, 65544, 131072, 128)])
def test_products(tg, M, N, K, group):
    """C, the codes or the decoded weights past 2^32 elements; small integers, bit by bit."""
    need(60)
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(HALF)
    bq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    groups = K // group
    bscale = (2.0 ** torch.randint(-3, 1, (groups, N), generator=g, device="cuda")).to(HALF)
    c = tg.gemm_w4(a, bq, bscale, N, group)
    rows, cols = some_rows(M, N), some_rows(N, K)
    W = ops64.w4_weight(bq[cols], bscale[:, cols], None, len(cols), K, group)
    assert torch.equal(c[:, cols], (a.double() @ W.T).to(HALF))
    if M * N > 2 ** 32:
        W = ops64.w4_weight(bq, bscale, None, N, K, group)
        assert torch.equal(c[rows], (a[rows].double() @ W.T).to(HALF))


@pytest.mark.parametrize("M", [1, 12, 40, 65, 300])
@pytest.mark.parametrize("dtype,scale", [(HALF, 2.0 ** -19), (HALF, 2.0 ** -23), (BF16, 2.0 ** -128)])
def test_subnormal_scales(tg, M, dtype, scale):
    """Rows of A with a single number: the result is a weight times it."""
    N, K, group = 520, 512, 32
    g = torch.Generator(device="cuda").manual_seed(M)
    bq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (scale * (1 + torch.rand(K // group, N, generator=g, device="cuda", dtype=torch.float64))).to(dtype)
    factor = 16.0 if dtype is HALF else 2.0 ** 100
    at = torch.arange(M, device="cuda") * 7 % K
    a = torch.zeros(M, K, device="cuda", dtype=dtype)
    a[torch.arange(M, device="cuda"), at] = factor
    want = factor * ops64.w4_weight(bq, s, None, N, K, group).T[at]
    c = tg.gemm_w4(a, bq, s, N, group, out_dtype=F32)
    assert torch.equal(c.double(), want)
