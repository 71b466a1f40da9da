"""The layer norm, the codes and their products together, as a served model and a training
step use them, on a GB300: queued without a wait, captured, on two streams, from two threads."""

import threading

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


class Block:
    """One block with layer norms and 8-bit weights."""

    def __init__(self, tg, dim, hidden, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.weight, self.bias = 1 + 0.1 * normal(dim), 0.1 * normal(dim)
        self.up = tg.quantize_rows(normal(hidden, dim) * dim ** -0.5)
        self.down = tg.quantize_rows(normal(dim, hidden) * hidden ** -0.5)
        self.up_bias = 0.1 * normal(hidden)

    def run(self, tg, o, stream, kept=None):
        """The block's output and its residual stream, from those of the block before."""
        y, a, sa = tg.layer_norm_i8(o, stream, weight=self.weight, bias=self.bias)
        f = tg.gemm_i8(a, self.up[0], sa, self.up[1], True, bias=self.up_bias, out_dtype=BF16)
        b, sb = tg.quantize_rows(f)
        out = tg.gemm_i8(b, self.down[0], sb, self.down[1], out_dtype=BF16)
        if kept is not None:
            kept.append((self, o, stream, y, a, sa, f, b, sb, out))
        return out, y


def check(kept):
    for block, o, stream, y, a, sa, f, b, sb, out in kept:
        norm = ref.LayerNorm(o, stream, weight=block.weight, bias=block.bias)
        norm.check(y, None, "y")
        norm.check_codes(a, sa, "codes")
        ref.assert_close(f, *ref.i8(a, block.up[0], sa, block.up[1], bias=block.up_bias, relu=True), "up")
        want = ref.codes_of(f)
        assert torch.equal(b, want[0]) and torch.equal(sb, want[1])
        ref.assert_close(out, *ref.i8(b, block.down[0], sb, block.down[1]), "down")


@pytest.mark.parametrize("tokens", [1, 5, 16, 50, 300])
@pytest.mark.parametrize("dim,hidden", [(512, 2048), (1000, 1303)])
def test_blocks_one_after_another(tg, tokens, dim, hidden):
    """Each step against its 64-bit form on what the step before gave; nothing waits in between."""
    blocks = [Block(tg, dim, hidden, s) for s in range(3)]
    g = torch.Generator(device="cuda").manual_seed(tokens)
    o = torch.randn(tokens, dim, generator=g, device="cuda").to(BF16)
    stream = torch.randn(tokens, dim, generator=g, device="cuda")
    kept = []
    for block in blocks:
        o, stream = block.run(tg, o, stream, kept)
    check(kept)


@pytest.mark.parametrize("tokens", [1, 12, 100])
def test_a_captured_stack(tg, tokens):
    """Captured once, replayed on new inputs: the bits of the eager calls."""
    blocks = [Block(tg, 640, 1920, s) for s in range(2)]
    x = torch.randn(tokens, 640, device="cuda").to(BF16)
    r = torch.randn(tokens, 640, device="cuda")

    def stack(o, stream):
        for block in blocks:
            o, stream = block.run(tg, o, stream)
        return tg.layer_norm(o, stream, weight=blocks[0].weight)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = stack(x, r)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(tokens, 640, generator=g, device="cuda"))
        r.copy_(torch.randn(tokens, 640, generator=g, device="cuda"))
        graph.replay()
        want = stack(x, r)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


def test_two_streams_at_once(tg):
    blocks = [Block(tg, 768, 2304, s) for s in range(2)]
    inputs = [(torch.randn(n, 768, device="cuda").to(BF16), torch.randn(n, 768, device="cuda"))
              for n in (70, 300)]
    want = [b.run(tg, *i) for b, i in zip(blocks, inputs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(blocks[k].run(tg, *inputs[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_two_threads_at_once(tg):
    block = Block(tg, 768, 2304, 5)
    inputs = [(torch.randn(n, 768, device="cuda").to(BF16), torch.randn(n, 768, device="cuda"))
              for n in (40, 200)]
    want = [block.run(tg, *i) for i in inputs]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                out = block.run(tg, *inputs[k])
                grads = tg.layer_norm_backward(None, out[0], inputs[k][0], weight=block.weight)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(out, want[k])) or not grads.x.isfinite().all():
                    bad.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("rows,dim", [(64, 256), (300, 1001)])
def test_a_training_step(tg, rows, dim):
    """Two norms with a product between them, the residual stream through both: the gradients
    against autograd in 64 bits.  In fp32: the products' sums lose at most dim·2^-24 of their
    size, the norms some (dim/32 + 32)·2^-23; two norms, two products and their gradients in a
    row: 2^-22·(dim + 64) of the results' size covers each by a factor above two."""
    g = torch.Generator(device="cuda").manual_seed(rows)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x, r, w = normal(rows, dim), normal(rows, dim), normal(dim, dim) * dim ** -0.5
    w1, b1, w2, b2 = 1 + 0.1 * normal(dim), 0.1 * normal(dim), 1 + 0.1 * normal(dim), 0.1 * normal(dim)
    dy, dh = normal(rows, dim), normal(rows, dim)
    y1, h1 = tg.layer_norm(x, r, weight=w1, bias=b1)
    o = h1 @ w
    y2, h2 = tg.layer_norm(o, y1, weight=w2, bias=b2)
    second = tg.layer_norm_backward(dy, dh, o, y1, weight=w2, bias=b2)
    first = tg.layer_norm_backward(second.residual, second.x @ w.T, x, r, weight=w1, bias=b1)
    leaves = [t.double().requires_grad_() for t in (x, r, w1, b1, w2, b2)]

    def norm(v, weight, bias):
        d = v - v.mean(dim=1, keepdim=True)
        return d * torch.rsqrt((d * d).mean(dim=1, keepdim=True) + 1e-5) * weight + bias

    a = leaves[0] + leaves[1]
    b = norm(a, leaves[2], leaves[3]) @ w.double() + a
    loss = (b * dy.double()).sum() + (norm(b, leaves[4], leaves[5]) * dh.double()).sum()
    want = torch.autograd.grad(loss, leaves)
    for got, exact in zip((first.x, first.residual, first.weight, first.bias, second.weight, second.bias), want):
        off = float((got.double() - exact).norm() / exact.norm())
        assert off <= (dim + 64) * 2.0 ** -22, off
