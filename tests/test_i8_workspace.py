"""What tg_gemm_i8 asks of its workspace: nothing where its kernel has none."""

import pytest


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    t.library()
    return t


@pytest.mark.parametrize("M,N,K", [(1, 40, 131071), (8, 28672, 4096), (9, 28672, 4096), (16, 4096, 28672),
                                   (16, 100000, 8192), (12, 1, 1), (32, 5000, 4096), (48, 1024, 1024),
                                   (64, 512, 1024), (20, 40, 0), (300, 40, 0)])
def test_none_for_few_rows(tg, M, N, K):
    assert tg.tg_gemm_i8_workspace(M, N, K) == 0


@pytest.mark.parametrize("M,N,K", [(16, 4096, 131071), (17, 28672, 4096), (33, 5000, 4096), (64, 4096, 4096),
                                   (65, 512, 1024), (512, 16384, 8192), (300, 300, 128)])
def test_some_for_the_others(tg, M, N, K):
    """A as fp16 at least, and no more than 48 MB besides."""
    rows = -(-K // 128) * 128 * M * 2
    assert rows <= tg.tg_gemm_i8_workspace(M, N, K) <= rows + (48 << 20)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(8, 300, 1000), (16, 300, 28672), (40, 1000, 1024), (20, 300, 0)])
@pytest.mark.parametrize("size", [0, 256])
def test_calls_with_less_than_the_other_kernel_needs(tg, M, N, K, size):
    """A workspace that holds nothing, or nearly: it is not written, in a capture neither."""
    torch = pytest.importorskip("torch")
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = (torch.randint(-9, 10, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    one = torch.ones(max(M, N), device="cuda")
    b = torch.nn.functional.pad(b, (0, -K % 16))
    want = (a.double() @ b[:, :K].double().T).float()
    work = torch.full((512,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, device="cuda")

    def call():
        epi = tg.tg_epilogue_ex_t(0, 2, None, None, 0)
        assert tg.tg_gemm_i8(a.data_ptr(), max(K, 1), one.data_ptr(), b.data_ptr(), b.shape[1], one.data_ptr(),
                             out.data_ptr(), N, M, N, K, epi, work.data_ptr(), size,
                             torch.cuda.current_stream().cuda_stream) == 0

    call()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((work == 0x5a).all())
    tg.sync_status()
