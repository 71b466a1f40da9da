"""tg_norm_residual and its gradient against their 64-bit forms on a GB300.

Tolerances: ops64.py (everything in fp32, each output rounded once).
"""

import pytest

import ops64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [(HALF, HALF), (BF16, BF16), (BF16, F32), (HALF, F32), (F32, F32)]


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def make(rows, cols, dtype, stream, *, residual=True, post=True, gates=1, pre=True, pad=0, seed=0,
         empty=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + 17 * rows + cols)

    def mat(r, kind, factor=1.0):
        whole = torch.randn(r, cols + pad, generator=g, device="cuda") * factor
        if empty:
            whole[r - empty:] = 0
        return whole.to(kind)[:, :cols]

    def vec():
        return 1.0 + 0.3 * torch.randn(cols, generator=g, device="cuda")

    x = mat(rows, dtype, 2.0)
    kept = dict(residual=mat(rows, stream, 3.0) if residual else None,
                post_weight=vec() if post else None,
                gate=torch.randn(gates, cols + pad, generator=g, device="cuda").to(dtype)[:, :cols]
                if gates else None,
                scale=0.6, pre_weight=vec() if pre else None, eps=1e-5)
    return x, kept, mat(rows, stream if residual else dtype), mat(rows, dtype) if pre else None


def check(tg, rows, cols, dtype, stream, **how):
    x, kept, dy, dh = make(rows, cols, dtype, stream, **how)
    ref = ops64.Norm(x, **kept)
    what = f"{rows}x{cols} {dtype} {stream} {how}"
    y, h = tg.norm_residual(x, **kept)
    assert y.dtype == (stream if kept["residual"] is not None else dtype)
    assert (h is None) == (kept["pre_weight"] is None)
    ref.check(y, h, what)
    grads = tg.norm_residual_backward(dy, dh, x, **kept)
    for got, inp in zip(grads, (x, kept["residual"], kept["gate"], kept["post_weight"],
                                kept["pre_weight"])):
        assert (got is None) == (inp is None)
        if got is not None:
            assert got.dtype == inp.dtype and got.shape == inp.shape
    ref.check_grads(grads, dy, dh, what)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("cols", [1, 7, 8, 32, 100, 256, 257, 768, 1000, 1024, 1025, 2048, 4096,
                                  5119, 8192, 12000, 16384, 16385, 20000, 32768])
def test_widths(tg, dtype, stream, cols):
    check(tg, 5, cols, dtype, stream)
    check(tg, 6, cols, dtype, stream, gates=2, pad=1, seed=1)


@pytest.mark.parametrize("rows", [1, 2, 3, 151, 152, 153, 303, 305, 1000, 2053])
@pytest.mark.parametrize("cols", [96, 1536])
def test_rows(tg, rows, cols):
    check(tg, rows, cols, BF16, F32)
    check(tg, rows, cols, HALF, HALF, gates=rows, pad=8, seed=2)


@pytest.mark.parametrize("rows,gates", [(1200, 2), (1200, 3), (1200, 100), (1200, 400), (1200, 600),
                                        (1200, 1200), (2000, 1000), (7, 7), (4000, 800)])
def test_gates(tg, rows, gates):
    check(tg, rows, 264, BF16, BF16, gates=gates)
    check(tg, rows, 65, F32, F32, gates=gates, pad=3)


@pytest.mark.parametrize("cols,pad", [(4097, 0), (4104, 8), (5121, 1), (9000, 0), (16392, 8), (30000, 3)])
@pytest.mark.parametrize("rows,gates", [(1, 1), (40, 40), (300, 3), (300, 100), (700, 1), (400, 200)])
def test_long_rows(tg, cols, pad, rows, gates):
    """Rows that several blocks share, with gates of one, some and all rows."""
    check(tg, rows, cols, torch.bfloat16, torch.float32, gates=gates, pad=pad)
    check(tg, rows, cols, torch.float16, torch.float16, gates=gates, pad=pad, post=rows != 300)


def test_a_wait_for_another_block_that_runs_out_is_reported_once(tg):
    """Values that are not sent: the gradient's kernel gives up within its limit and
    returns, the status says so once, and the next call is right."""
    x, kept, dy, dh = make(3, 9000, torch.bfloat16, torch.bfloat16)
    want = tg.norm_residual_backward(dy, dh, x, **kept)
    tg.sync_status()
    try:
        tg.tg_debug_set_wait_timeout_ns(20_000_000)
        tg.tg_debug_inject(1)
        tg.norm_residual_backward(dy, dh, x, **kept)
        with pytest.raises(tg.TgemmError) as e:
            tg.sync_status()
        assert e.value.status == tg.TG_ERR_TIMEOUT
        tg.sync_status()
    finally:
        tg.tg_debug_inject(0)
        tg.tg_debug_set_wait_timeout_ns(0)
    for a, b in zip(tg.norm_residual_backward(dy, dh, x, **kept), want):
        assert torch.equal(a, b)
    tg.sync_status()


@pytest.mark.parametrize("rows,gates", [(1, 1), (6, 0), (6, 3)])
def test_plain_and_general_calls_agree(tg, rows, gates):
    """A call whose results are given takes another way through the binding: the same bits."""
    x, kept, dy, dh = make(rows, 520, torch.bfloat16, torch.float32, gates=gates)
    y, h = tg.norm_residual(x, **kept)
    other = tg.norm_residual(x, out=torch.empty_like(y), normed=torch.empty_like(h), **kept)
    assert torch.equal(y, other[0]) and torch.equal(h, other[1])
    grads = tg.norm_residual_backward(dy, dh, x, **kept)
    assert isinstance(grads, tg.NormGrads)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for a, b in zip(grads, tg.norm_residual_backward(dy, dh, x, stream=stream, **kept)):
        stream.synchronize()
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    weight = torch.nn.Parameter(kept["pre_weight"])
    again = tg.norm_residual(x, **dict(kept, pre_weight=weight))
    assert torch.equal(again[1], h) and not again[1].requires_grad


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gates", [0, 1])
@pytest.mark.parametrize("pre", [True, False])
def test_parts(tg, residual, post, gates, pre):
    for cols in (200, 1024, 17000):
        check(tg, 33, cols, BF16, F32 if residual else BF16, residual=residual, post=post,
              gates=gates, pre=pre)


@pytest.mark.parametrize("cols", [130, 4096, 18000])
def test_missing_gradients_are_zero(tg, cols):
    x, kept, dy, dh = make(40, cols, BF16, F32)
    ref = ops64.Norm(x, **kept)
    ref.check_grads(tg.norm_residual_backward(None, dh, x, **kept), None, dh, "no dy")
    only = tg.norm_residual_backward(dy, None, x, **kept)
    ref.check_grads(only, dy, None, "no dh")
    assert not bool(only.pre_weight.any())
    for g in tg.norm_residual_backward(None, None, x, **kept):
        assert not bool(g.any())


@pytest.mark.parametrize("cols", [64, 4096, 17000])
def test_rows_of_zeros(tg, cols):
    """Padding rows: the statistics rest on eps alone, nothing becomes NaN."""
    x, kept, dy, dh = make(64, cols, HALF, F32, empty=20)
    y, h = tg.norm_residual(x, **kept)
    assert not bool(y[44:].any()) and not bool(h[44:].any())
    grads = tg.norm_residual_backward(dy, dh, x, **kept)
    ref = ops64.Norm(x, **kept)
    ref.check(y, h)
    ref.check_grads(grads, dy, dh)
    assert not bool(grads.x[44:].any()) and not bool(grads.residual[44:].any())


@pytest.mark.parametrize("cols", [96, 2048, 17000])
def test_nan_and_infinity_stay_in_their_row(tg, cols):
    x, kept, dy, dh = make(50, cols, BF16, BF16)
    y0, h0 = tg.norm_residual(x, **kept)
    g0 = tg.norm_residual_backward(dy, dh, x, **kept)
    x = x.clone()
    x[3, 5], x[9, cols - 1] = float("nan"), float("inf")
    y, h = tg.norm_residual(x, **kept)
    g = tg.norm_residual_backward(dy, dh, x, **kept)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[[3, 9]] = False
    for a, b in ((y, y0), (h, h0), (g.x, g0.x), (g.residual, g0.residual)):
        assert torch.equal(a[keep], b[keep])
    assert bool(h[3].isnan().all())
    assert bool(h[9, cols - 1].isnan()) and bool(y[9, cols - 1].isnan())


@pytest.mark.parametrize("cols", [300, 4096, 9000, 20000])
def test_sum_in_place(tg, cols):
    x, kept, _, _ = make(21, cols, BF16, F32)
    want = tg.norm_residual(x, **kept)
    r = kept["residual"]
    got = tg.norm_residual(x, **kept, out=r)
    assert got[0] is r and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cols", [200, 2048, 17000])
def test_outputs_keep_to_their_columns(tg, cols):
    x, kept, _, _ = make(9, cols, HALF, HALF, pad=5)
    whole = [torch.full((9, cols + 3), 7.0, device="cuda", dtype=HALF) for _ in range(2)]
    y, h = tg.norm_residual(x, **kept, out=whole[0][:, :cols], normed=whole[1][:, :cols])
    ops64.Norm(x, **kept).check(y, h)
    for w in whole:
        assert bool((w[:, cols:] == 7.0).all())


def test_gradient_against_differences(tg):
    """The change of L = Σ y·dy + Σ h·dh along a direction, by central differences of
    the 64-bit forward form, against the kernel's gradient in fp32 inputs."""
    for rows, cols, gates in ((6, 40, 1), (8, 300, 2), (4, 1024, 4)):
        x, kept, dy, dh = make(rows, cols, F32, F32, gates=gates)
        names = ("x", "residual", "gate", "post_weight", "pre_weight")
        at = dict(x=x, **{k: kept[k] for k in names[1:]})
        grads = tg.norm_residual_backward(dy, dh, x, **kept)
        g = torch.Generator(device="cuda").manual_seed(3)

        def loss(point):
            ref = ops64.Norm(point["x"], **{**kept, **{k: point[k] for k in names[1:]}})
            return float((ref.y * dy.double()).sum() + (ref.h * dh.double()).sum())

        for name, grad in zip(names, grads):
            v = torch.randn(at[name].shape, generator=g, device="cuda", dtype=torch.float64)
            step = 1e-5
            hi, lo = (dict({k: t.double() for k, t in at.items()}, **{
                name: at[name].double() + sign * step * v}) for sign in (1, -1))
            slope = (loss(hi) - loss(lo)) / (2 * step)
            mine = float((grad.double() * v).sum())
            size = float((grad.double() * v).abs().sum())
            # differences: step² of the third derivative and 2^-53 · L / step, both
            # below 1e-8 of the size; the gradient: fp32, 1e-5 of the size at most
            assert abs(slope - mine) <= 2e-5 * size, (name, slope, mine, size)


def test_same_bits_every_time_and_on_another_stream(tg):
    for rows, cols, gates in ((700, 1024, 2), (64, 4096, 1), (300, 333, 300)):
        x, kept, dy, dh = make(rows, cols, BF16, F32, gates=gates)
        first = (*tg.norm_residual(x, **kept), *tg.norm_residual_backward(dy, dh, x, **kept))
        again = (*tg.norm_residual(x, **kept), *tg.norm_residual_backward(dy, dh, x, **kept))
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        there = (*tg.norm_residual(x, **kept, stream=other),
                 *tg.norm_residual_backward(dy, dh, x, **kept, stream=other))
        torch.cuda.current_stream().wait_stream(other)
        for a, b, c in zip(first, again, there):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_in_a_graph(tg):
    x, kept, dy, dh = make(500, 768, BF16, F32, gates=2)
    want = (*tg.norm_residual(x, **kept), *tg.norm_residual_backward(dy, dh, x, **kept))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tg.norm_residual_backward(dy, dh, x, **kept)  # the stream's workspace
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = (*tg.norm_residual(x, **kept), *tg.norm_residual_backward(dy, dh, x, **kept))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_no_workspace_inside_a_capture(tg):
    """A stream's first call in a capture is refused, and the capture goes on."""
    x, kept, dy, dh = make(50, 256, BF16, F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(tg.TgemmError) as e:
            tg.norm_residual_backward(dy, dh, x, **kept)
        y, h = tg.norm_residual(x, **kept)
    assert e.value.status == tg.TG_ERR_NO_MEMORY
    graph.replay()
    torch.cuda.synchronize()
    ops64.Norm(x, **kept).check(y, h)


def test_no_rows(tg):
    x, kept, dy, dh = make(0, 64, BF16, F32, gates=0)
    y, h = tg.norm_residual(x, **kept)
    assert y.shape == h.shape == (0, 64)
    g = tg.norm_residual_backward(dy, dh, x, **kept)
    assert g.x.shape == (0, 64)
    assert not bool(g.post_weight.any()) and not bool(g.pre_weight.any())
    kept["gate"] = torch.ones(64, device="cuda", dtype=BF16)
    assert not bool(tg.norm_residual_backward(dy, dh, x, **kept).gate.any())


def test_refusals(tg):
    x, kept, dy, dh = make(6, 64, BF16, F32)
    bad = [
        (TypeError, dict(x=x.double())),
        (ValueError, dict(x=x.t())),
        (ValueError, dict(x=x.cpu())),
        (TypeError, dict(residual=kept["residual"].to(HALF))),
        (ValueError, dict(residual=kept["residual"][:5])),
        (ValueError, dict(post_weight=kept["post_weight"][:63])),
        (ValueError, dict(post_weight=kept["post_weight"].to(BF16))),
        (ValueError, dict(pre_weight=kept["pre_weight"].cpu())),
        (TypeError, dict(gate=kept["gate"].float())),
        (ValueError, dict(gate=kept["gate"].expand(4, 64).contiguous())),
        (ValueError, dict(gate=kept["gate"][:, :63])),
        (ValueError, dict(eps=-1.0)),
        (ValueError, dict(eps=float("nan"))),
    ]
    for kind, change in bad:
        with pytest.raises(kind):
            tg.norm_residual(**{**dict(x=x, **kept), **change})
        with pytest.raises(kind):
            tg.norm_residual_backward(dy, dh, **{**dict(x=x, **kept), **change})
    for kind, change in ((TypeError, dict(out=x.clone())), (ValueError, dict(out=dy[:5])),
                         (TypeError, dict(normed=dy))):
        with pytest.raises(kind):
            tg.norm_residual(x, **kept, **change)
    with pytest.raises(ValueError):
        tg.norm_residual(x, **{**kept, "pre_weight": None}, normed=dh)
    with pytest.raises(ValueError):
        tg.norm_residual_backward(dy, dh, x, **{**kept, "pre_weight": None})
    with pytest.raises(TypeError):
        tg.norm_residual_backward(dy.to(BF16), dh, x, **kept)
    with pytest.raises(ValueError):
        tg.norm_residual(torch.zeros(2, 32769, device="cuda"))
    with pytest.raises(tg.TgemmError) as e:
        tg.norm_residual(x[:1].expand(6, 64), **kept)  # row stride 0
    assert e.value.status == tg.TG_ERR_INVALID_VALUE
