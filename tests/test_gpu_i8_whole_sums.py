"""The sums of tg_gemm_i8 are whole numbers at every size: with unit scales and fp32 results each
is the sum itself, rounded once.  K, N and M are those at which the accumulators have to give
their sums away in mid-row, on both sides of each choice between kernels."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    yield t
    t.sync_status()


def ints(rows, cols, low, high, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole = torch.randint(low, high, (rows, (cols + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.int8)
    return whole[:, :cols]


def sums(a, b):
    """a @ b.T, exactly: 512 products of at most 2^14 are exact in fp32, and their sums in 64 bits."""
    assert not torch.backends.cuda.matmul.allow_tf32
    c = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 512):
        c += a[:, k:k + 512].float() @ b[:, k:k + 512].float().T
    return c


def product(tg, a, b):
    one = torch.ones(max(a.shape[0], b.shape[0]), device=a.device)
    return tg.gemm_i8(a, b, one[:a.shape[0]], one[:b.shape[0]], out_dtype=torch.float32)


def check(tg, a, b, rows):
    want = sums(a, b).float()  # (rounded once)
    for m in rows:
        got = product(tg, a[:m], b)
        assert torch.equal(got, want[:m]), (m, float((got - want[:m]).abs().max()))


ROWS = (1, 7, 8, 9, 12, 16, 17, 24, 32, 33, 48, 64, 65, 100, 129, 256, 300)


@pytest.mark.parametrize("N,K", [(300, 28672), (300, 131071), (4096, 8192), (2500, 28672), (19456, 8192),
                                 (30000, 2100), (19500, 4099)])
def test_halves_that_cancel(tg, N, K):
    """A first half of large sums, a second half that takes them back."""
    a = ints(300, K, 60, 128, 1)
    b = ints(N, K, 60, 128, 2)
    b[:, K // 2:] *= -1
    check(tg, a, b, ROWS)
    a[:, 1:K // 2] = 127
    b[:, 1:K // 2] = 127
    a[:, K - K // 2 + 1:] = 127
    b[:, K - K // 2 + 1:] = -127
    check(tg, a, b, (16, 17, 64, 256, 300))


@pytest.mark.parametrize("N,K", [(200, 131071), (1000, 28672), (640, 8192), (19456, 4096), (6000, 20000),
                                 (128, 1032), (20000, 1160), (600, 8192), (100, 9001), (3600, 8200)])
def test_any_codes(tg, N, K):
    """Few rows of long and of wide weights among them, whose sums are 32-bit numbers from the start:
    no code may be lost, however small its part of a sum."""
    check(tg, ints(300, K, -128, 128, 3), ints(N, K, -128, 128, 4), ROWS)


@pytest.mark.parametrize("value", [(127, 127), (-128, -128), (-128, 127), (127, 126)])
@pytest.mark.parametrize("N,K", [(20, 131071), (20, 1040), (19456, 2049), (600, 28672)])
def test_largest_codes(tg, N, K, value):
    """All products of one sign and size: as many units as fit below 2^24, and not one more."""
    a = torch.full((300, K), value[0], dtype=torch.int8, device="cuda")
    b = ints(N, K, 0, 1, 0)
    b.fill_(value[1])
    want = torch.tensor(float(K * value[0] * value[1]), dtype=torch.float64).float().item()
    for m in (1, 8, 16, 17, 64, 200, 300):
        assert bool((product(tg, a[:m], b) == want).all()), m


@pytest.mark.parametrize("M", [20, 70, 256, 300])
def test_one_token_of_large_codes(tg, M):
    """The largest codes are one token's, in the last columns, the first ones, or nowhere."""
    K, N = 9001, 2000
    b = ints(N, K, 90, 128, 5)
    b[:, 4500:] *= -1
    for where in (slice(0, 5000), slice(4000, K), slice(0, 0)):
        a = ints(M, K, -1, 2, 6)
        a[M - 1, where] = ints(1, K, 90, 128, 7)[0, where]
        check(tg, a, b, (M,))
    a = ints(M, K, 0, 1, 8)  # zeros
    check(tg, a, b, (M,))


def test_more_rows_than_a_slab(tg):
    """A has more rows than are taken at a time; the large codes are in the second part."""
    K, M = 28672, 18900
    a = ints(M, K, -1, 2, 9)
    a[-40:] = ints(40, K, 100, 128, 10)
    b = ints(24, K, 100, 128, 11)
    b[:, K // 2:] *= -1
    check(tg, a, b, (M,))


@pytest.mark.parametrize("M", [33, 256, 700])
@pytest.mark.parametrize("N,K", [(19456, 4099), (5000, 12000), (300, 28672)])
def test_the_same_bits_with_an_epilogue_and_any_workspace(tg, M, N, K):
    """Sums that leave the accumulator several times, into given rows, from a workspace that held
    something else, over and over."""
    a, b = ints(M, K, 60, 128, 12), ints(N, K, -128, 128, 13)
    sa, sb = torch.rand(M, device="cuda") / 1000 + 0.001, torch.rand(N, device="cuda") / 1000 + 0.001
    bias = torch.randn(N, device="cuda") * 10
    r = torch.randn(M, N, device="cuda")
    v = sums(a, b).float().double() * sa[:, None].double() * sb.double()
    # the sum is rounded; then each scale, the bias and the residual round once more
    bound = 2.0 ** -24 * (4 * v.abs() + 2 * bias.double().abs() + 2 * r.double().abs())
    v = v + bias.double()
    want, first = torch.where(v > 0, v, torch.zeros_like(v)) + r.double(), None
    size = tg.tg_gemm_i8_workspace(M, N, K)
    work = torch.full((size,), 0xa5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out = r.clone()
        epi = tg.tg_epilogue_ex_t(1, 2, bias.data_ptr(), out.data_ptr(), N)
        st = tg.tg_gemm_i8(a.data_ptr(), a.stride(0), sa.data_ptr(), b.data_ptr(), b.stride(0), sb.data_ptr(),
                           out.data_ptr(), N, M, N, K, epi, work.data_ptr(), size,
                           torch.cuda.current_stream().cuda_stream)
        assert st == 0 and bool(((out.double() - want).abs() <= bound).all())
        assert first is None or torch.equal(out, first)
        first = out
