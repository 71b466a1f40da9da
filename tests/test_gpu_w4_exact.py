"""tg_gemm_w4 bit by bit on a GB300, at the sizes of layers.

The bounds of test_gpu_w4.py grow with K: at some thousand k they would pass a product that
leaves out a group, or rounds its weights.  Here no bound is needed:

- small integers with scales that are powers of two.  Every term is a multiple of 1/8 and at
  most 30, its sign as likely one as the other: sums of any of a row's terms are some thousands
  (5·sqrt(K)), far below the 2^21 up to which fp32 holds them exactly.  So every order of
  summation gives the exact result, which is then rounded once;
- rows of A with a single one: the result is a weight.
"""

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KINDS = [(HALF, 128, False), (BF16, 32, True), (HALF, 64, True)]


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def up(n, to):
    return -(-n // to) * to


def weights(N, K, dtype, group, zeros, g, scales):
    groups = up(K, group) // group
    bq = torch.randint(0, 256, (N, up((K + 1) // 2, 16)), generator=g, device="cuda",
                       dtype=torch.uint8)[:, :(K + 1) // 2]
    bscale = scales(groups, up(N, 8)).to(dtype)[:, :N]
    bzero = None
    if zeros:
        bzero = torch.randint(0, 16, (groups, up(N, 16)), generator=g, device="cuda",
                              dtype=torch.uint8)[:, :N]
    return bq, bscale, bzero


def check_integers(tg, M, N, K, dtype, group, zeros, pad=0):
    g = torch.Generator(device="cuda").manual_seed(M + 31 * N + 101 * K + group)
    bq, bscale, bzero = weights(
        N, K, dtype, group, zeros, g,
        lambda r, c: 2.0 ** torch.randint(-3, 1, (r, c), generator=g, device="cuda").float())
    a = torch.randint(-2, 3, (M, K + pad), generator=g, device="cuda").to(dtype)[:, :K]
    want = a.double() @ ops64.w4_weight(bq, bscale, bzero, N, K, group).T
    assert float(want.abs().max()) < 2 ** 16
    for out_dtype in (None, F32):
        c = tg.gemm_w4(a, bq, bscale, N, group, bzero=bzero, out_dtype=out_dtype)
        assert torch.equal(c, want.to(c.dtype)), f"{int((c != want.to(c.dtype)).sum())} of {c.numel()}"
    tg.sync_status()


@pytest.mark.parametrize("dtype,group,zeros", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 28672, 4096), (1, 4096, 28672), (8, 16384, 8192), (16, 4096, 28672),
                                   (33, 16384, 8192), (64, 16384, 8192), (65, 16384, 8192),
                                   (200, 16384, 8192), (512, 16384, 8192), (700, 4096, 28672),
                                   (7000, 16384, 8192), (4096, 512, 2048)])
def test_integers_at_layer_sizes(tg, M, N, K, dtype, group, zeros):
    """The last two take the way over decoded weights with a 16-bit result."""
    check_integers(tg, M, N, K, dtype, group, zeros)


@pytest.mark.parametrize("dtype,group,zeros", KINDS)
@pytest.mark.parametrize("M,N,K", [(7, 5003, 4099), (50, 2311, 9001), (130, 1031, 20001), (513, 777, 4097),
                                   (8, 40, 100001), (16, 33, 60001), (3, 20, 700001), (11, 20, 600001),
                                   (70, 20, 300001)])
def test_integers_at_odd_sizes(tg, M, N, K, dtype, group, zeros):
    """Among them k too long for 8 or 16 rows of A in a cluster's shared memory, and for one."""
    check_integers(tg, M, N, K, dtype, group, zeros, pad=1)


@pytest.mark.parametrize("dtype,group,zeros", KINDS)
@pytest.mark.parametrize("M", [1, 9, 40, 64, 65, 300, 1000])
def test_a_single_one_gives_a_weight(tg, M, dtype, group, zeros):
    """An fp32 result is the weight itself, with none of its up to 15 bits lost; a 16-bit
    result is the weight rounded."""
    N, K = 4100, 4096
    g = torch.Generator(device="cuda").manual_seed(M)
    bq, bscale, bzero = weights(N, K, dtype, group, zeros, g,
                                lambda r, c: 0.01 * (1 + torch.rand(r, c, generator=g, device="cuda")))
    at = torch.randperm(K, generator=g, device="cuda")[:M]
    a = torch.zeros(M, K, device="cuda", dtype=dtype)
    a[torch.arange(M, device="cuda"), at] = 1
    want = ops64.w4_weight(bq, bscale, bzero, N, K, group).T[at]
    for out_dtype in (None, F32):
        c = tg.gemm_w4(a, bq, bscale, N, group, bzero=bzero, out_dtype=out_dtype)
        assert torch.equal(c, want.to(c.dtype))
    tg.sync_status()


@pytest.mark.parametrize("M,N,K,decoded", [(100, 512, 2048, False), (257, 600, 4096, False), (1500, 512, 4096, False),
                                           (5000, 512, 4096, True), (6000, 1024, 1024, True)])
def test_which_products_decode_their_weights_to_memory(tg, M, N, K, decoded):
    """Those of very many rows: their product is a dense GEMM launch."""
    a = torch.zeros(M, K, device="cuda", dtype=HALF)
    bq = torch.zeros(N, K // 2, device="cuda", dtype=torch.uint8)
    scale = torch.ones(K // 128, N, device="cuda", dtype=HALF)
    x = torch.zeros(8, 8, device="cuda", dtype=HALF)
    tg.gemm(x, x)
    before = tg.tg_debug_last_launch()
    tg.gemm_w4(a, bq, scale, N, 128)
    after = tg.tg_debug_last_launch()
    assert (bytes(after) != bytes(before)) == decoded


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (5, 4096, 8192), (8, 8192, 4096), (16, 1024, 4096),
                                   (40, 512, 2048)])
@pytest.mark.parametrize("dtype,group,zeros", KINDS)
def test_weights_in_turn(tg, M, N, K, dtype, group, zeros):
    """Two weights in turn, again and again: a stage of a warp's ring that is filled again
    before all lanes have read it would show in some sum."""
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(dtype)
    both = [weights(N, K, dtype, group, zeros, g,
                    lambda r, c: 2.0 ** torch.randint(-3, 1, (r, c), generator=g, device="cuda").float())
            for _ in range(2)]
    want = [(a.double() @ ops64.w4_weight(*w, N, K, group).T).float() for w in both]
    got = [tg.gemm_w4(a, bq, s, N, group, bzero=z, out_dtype=F32) for _ in range(25) for bq, s, z in both]
    for i, c in enumerate(got):
        assert torch.equal(c, want[i % 2])
