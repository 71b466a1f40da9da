"""The 4-bit products after a wait that ran out and was reported, on a GB300: captured graphs
and calls that follow are right.  (Tiles that blocks share are counted in the stream's
workspace, and a launch that gives up leaves its counts there.)"""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


#: rows of A, N, K, result: kernels whose blocks share tiles
SHAPES = [(40, 4096, 4096, torch.half), (16, 1024, 16384, torch.half), (100, 512, 8192, torch.float32)]


class Case:
    """A product on a stream of its own, its weights fixed, its A a buffer."""

    def __init__(self, tg, M, N, K, out_dtype):
        self.tg, self.shape = tg, (M, N, K)
        g = torch.Generator(device="cuda").manual_seed(K)
        self.g = g
        self.bq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scale = torch.full((K // 64, N), 0.01, device="cuda", dtype=torch.half)
        self.a = torch.zeros(M, K, device="cuda", dtype=torch.half)
        self.out = torch.zeros(M, N, device="cuda", dtype=out_dtype)
        self.stream = torch.cuda.Stream()
        self.fresh()
        self.call()

    def call(self):
        self.tg.gemm_w4(self.a, self.bq, self.scale, self.shape[1], 64, out=self.out, stream=self.stream)
        self.stream.synchronize()

    def fresh(self):
        """Another A, and what the product with it is (from another stream's workspace)."""
        self.a.copy_(torch.randn(self.a.shape, generator=self.g, device="cuda"))
        self.want = self.tg.gemm_w4(self.a, self.bq, self.scale, self.shape[1], 64, out_dtype=self.out.dtype)
        self.out.zero_()
        torch.cuda.synchronize()

    def capture(self):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=self.stream):
            self.tg.gemm_w4(self.a, self.bq, self.scale, self.shape[1], 64, out=self.out)
        return graph

    def replay(self, graph):
        with torch.cuda.stream(self.stream):
            graph.replay()
        self.stream.synchronize()

    def check(self):
        assert torch.equal(self.out, self.want)
        self.tg.sync_status()


def run_out(tg, f):
    """f() with its first fetch left out and short waits; the report comes once."""
    tg.sync_status()
    try:
        tg.tg_debug_set_wait_timeout_ns(20_000_000)
        tg.tg_debug_inject(1)
        got = f()
    finally:
        tg.tg_debug_inject(0)
        tg.tg_debug_set_wait_timeout_ns(0)
    return got


def reported(tg):
    with pytest.raises(tg.TgemmError) as e:
        tg.sync_status()
    assert e.value.status == tg.TG_ERR_TIMEOUT
    tg.sync_status()


@pytest.mark.parametrize("shape", SHAPES)
def test_a_graph_captured_before(tg, shape):
    c = Case(tg, *shape)
    graph = c.capture()
    run_out(tg, c.call)
    reported(tg)
    for _ in range(3):
        c.fresh()
        c.replay(graph)
        c.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_a_call_after_one_that_was_only_captured(tg, shape):
    c = Case(tg, *shape)
    run_out(tg, c.call)
    reported(tg)
    c.capture()  # never replayed
    for _ in range(3):
        c.fresh()
        c.call()
        c.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_a_buffer_that_became_too_small(tg, shape):
    """Graphs keep the buffer that they were captured with."""
    c = Case(tg, *shape)
    graph = c.capture()
    gives_up = run_out(tg, c.capture)  # its launches withhold a fetch, at every replay
    big = torch.zeros(512, 16384, device="cuda", dtype=torch.half)
    bq = torch.zeros(16384, 8192, device="cuda", dtype=torch.uint8)
    scale = torch.ones(256, 16384, device="cuda", dtype=torch.half)
    tg.gemm_w4(big, bq, scale, 16384, 64, stream=c.stream)  # a larger one
    c.stream.synchronize()
    c.replay(gives_up)
    reported(tg)
    for _ in range(2):
        c.fresh()
        c.replay(graph)
        c.check()
