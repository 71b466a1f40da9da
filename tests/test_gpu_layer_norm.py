"""The layer norm, its codes and its gradient against their 64-bit forms on a GB300.

Tolerances: ops64_layer.py (everything in fp32, each output rounded once).
"""

import pytest

import ops64_layer as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [(HALF, HALF), (BF16, BF16), (BF16, F32), (HALF, F32), (F32, F32)]
WIDTHS = [1, 2, 7, 8, 9, 32, 100, 255, 256, 257, 768, 1000, 1024, 1025, 2040, 2048, 4096, 4104, 5119,
          8192, 8200, 12000, 16384, 16385, 20000, 32768, 32776]


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def make(rows, cols, dtype, stream, *, residual=True, weight=True, bias=True, pad=0, seed=0, empty=0,
         offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + 17 * rows + cols)

    def mat(kind, factor=1.0, offset=0.0):
        whole = torch.randn(rows, cols + pad, generator=g, device="cuda") * factor + offset
        if empty:
            whole[rows - empty:] = 0
        return whole.to(kind)[:, :cols]

    def vec(base):
        return base + 0.3 * torch.randn(cols, generator=g, device="cuda")

    x = mat(dtype, 2.0, offset)
    kept = dict(residual=mat(stream, 3.0) if residual else None, weight=vec(1.0) if weight else None,
                bias=vec(0.0) if bias else None, eps=1e-5)
    return x, kept, mat(stream if residual else dtype), mat(dtype)


def check(tg, rows, cols, dtype, stream, **how):
    x, kept, dy, dh = make(rows, cols, dtype, stream, **how)
    want = ref.LayerNorm(x, **kept)
    what = f"{rows}x{cols} {dtype} {stream} {how}"
    y, h = tg.layer_norm(x, **kept)
    assert h.dtype == dtype and h.shape == x.shape
    if kept["residual"] is None:
        assert y is None
    else:
        assert y.dtype == stream
    want.check(y, h, what)
    y2, codes, scale = tg.layer_norm_i8(x, **kept)
    assert (y2 is None) == (y is None) and (y is None or torch.equal(y, y2))
    want.check_codes(codes, scale, what)
    grads = tg.layer_norm_backward(dy, dh, x, **kept)
    for got, inp in zip(grads, (x, kept["residual"], kept["weight"], kept["bias"])):
        assert (got is None) == (inp is None)
        if got is not None:
            assert got.dtype == inp.dtype and got.shape == inp.shape
    want.check_grads(grads, dy, dh, what)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("cols", WIDTHS)
def test_widths(tg, dtype, stream, cols):
    check(tg, 5, cols, dtype, stream)
    check(tg, 6, cols, dtype, stream, pad=1, seed=1)
    check(tg, 3, cols, dtype, dtype, residual=False, pad=8, seed=2)


@pytest.mark.parametrize("cols", [65536, 131071])
def test_longest_rows(tg, cols):
    check(tg, 3, cols, BF16, F32)
    check(tg, 2, cols, F32, F32, pad=5)


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 151, 152, 153, 303, 305, 1000, 2053])
@pytest.mark.parametrize("cols", [96, 1536, 4096])
def test_rows(tg, rows, cols):
    check(tg, rows, cols, BF16, F32)
    check(tg, rows, cols, HALF, HALF, pad=8, seed=2)


@pytest.mark.parametrize("rows,cols,pad", [(40, 4104, 0), (300, 5121, 1), (700, 9000, 0), (400, 16392, 8),
                                           (170, 30000, 3), (20, 40000, 0)])
def test_long_rows(tg, rows, cols, pad):
    check(tg, rows, cols, BF16, F32, pad=pad)
    check(tg, rows, cols, HALF, HALF, pad=pad, bias=False)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_parts(tg, residual, weight, bias):
    for cols in (200, 1024, 17000):
        check(tg, 33, cols, BF16, F32 if residual else BF16, residual=residual, weight=weight, bias=bias)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("offset", [20.0, -3000.0])
def test_mean_far_from_zero(tg, dtype, stream, offset):
    for cols in (100, 1024, 4096, 9001):
        check(tg, 40, cols, dtype, stream, offset=offset)


def test_padding_rows(tg):
    """Rows of zeros: no deviation; h is the bias, its codes those of the bias."""
    check(tg, 50, 1024, BF16, F32, empty=13)
    x, kept, dy, dh = make(4, 512, HALF, HALF, empty=4, weight=False, bias=False)
    _, codes, scale = tg.layer_norm_i8(x, **kept)
    assert not bool(codes.any()) and not bool(scale.any())


@pytest.mark.parametrize("cols", [130, 1024, 4096, 18000])
def test_missing_gradients_are_zero(tg, cols):
    x, kept, dy, dh = make(40, cols, BF16, F32)
    want = ref.LayerNorm(x, **kept)
    want.check_grads(tg.layer_norm_backward(None, dh, x, **kept), None, dh, "no dy")
    got = tg.layer_norm_backward(dy, None, x, **kept)
    assert torch.equal(got.residual, dy) and torch.equal(got.x, dy.to(BF16))
    assert not bool(got.weight.any()) and not bool(got.bias.any())
    got = tg.layer_norm_backward(None, None, x, **kept)
    assert not any(bool(t.any()) for t in got)


@pytest.mark.parametrize("cols", [64, 2048, 9000])
def test_without_dh_values_need_not_be_finite(tg, cols):
    x, kept, dy, _ = make(5, cols, BF16, F32)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    got = tg.layer_norm_backward(dy, None, x, **kept)
    assert torch.equal(got.residual, dy)


@pytest.mark.parametrize("cols", [40, 256, 1000, 4096, 9000, 40000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_without_a_value(tg, cols, bad):
    """A NaN or an infinity makes its own row NaN, and no other."""
    for dtype, stream in ((BF16, F32), (HALF, HALF)):
        x, kept, dy, dh = make(6, cols, dtype, stream)
        clean = tg.layer_norm(x, **kept)
        ok = tg.layer_norm_backward(dy, dh, x, **kept)
        x[2, cols // 2] = bad
        y, h = tg.layer_norm(x, **kept)
        assert bool(h[2].isnan().all())
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(h[keep], clean[1][keep]) and torch.equal(y[keep], clean[0][keep])
        _, codes, scale = tg.layer_norm_i8(x, **kept)
        assert bool(scale[2].isnan()) and not bool(codes[2].any()) and bool(scale[keep].isfinite().all())
        got = tg.layer_norm_backward(dy, dh, x, **kept)
        assert bool(got.x[2].isnan().all()) and torch.equal(got.x[keep], ok.x[keep])
        assert bool(got.weight.isnan().all()) and torch.equal(got.bias, ok.bias)


@pytest.mark.parametrize("cols", [1, 257, 1024, 4096, 9000, 33000])
def test_the_sum_in_the_residuals_place(tg, cols):
    for pad in (0, 3):
        x, kept, _, _ = make(9, cols, BF16, F32, pad=pad)
        y, h = tg.layer_norm(x, **kept)
        y1, codes, scale = tg.layer_norm_i8(x, **kept)
        r = kept["residual"].clone()
        got = tg.layer_norm(x, **dict(kept, residual=r), out=r)
        assert got[0] is r and torch.equal(r, y) and torch.equal(got[1], h)
        r = kept["residual"].clone()
        got = tg.layer_norm_i8(x, **dict(kept, residual=r), out=r)
        assert torch.equal(r, y) and torch.equal(got[1], codes) and torch.equal(got[2], scale)


def test_nothing_past_the_rows_is_written(tg):
    """Results with wider rows: what lies between and behind them stays."""
    for cols in (64, 1000, 5000):
        x, kept, _, _ = make(7, cols, HALF, F32)
        want = tg.layer_norm(x, **kept)
        whole = [torch.full((9, cols + 5), 7.0, dtype=k, device="cuda") for k in (F32, HALF)]
        y, h = (w[1:8, 2:2 + cols] for w in whole)
        tg.layer_norm(x, **kept, out=y, normed=h)
        assert torch.equal(y, want[0])  # one addition
        # (h's sums may be taken in another order where rows lie otherwise: the bound of each)
        ref.LayerNorm(x, **kept).check(y, h, f"{cols}")
        for w in whole:
            assert bool((w[0] == 7).all() and (w[8] == 7).all() and (w[:, :2] == 7).all())
            assert bool((w[:, 2 + cols:] == 7).all())


@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("cols", [0, 5])
def test_no_rows_or_columns(tg, rows, cols):
    x, r = torch.ones(rows, cols, device="cuda"), torch.ones(rows, cols, device="cuda")
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    y, h = tg.layer_norm(x, r, weight=w, bias=b)
    assert y.shape == h.shape == x.shape
    y, codes, scale = tg.layer_norm_i8(x, r, weight=w, bias=b)
    assert codes.shape == x.shape and scale.shape == (rows,) and not bool(scale.any())
    codes, scale = tg.quantize_rows(x)
    assert codes.shape == x.shape and scale.shape == (rows,) and bool((scale == (1 / 127 if cols else 0)).all())
    g = tg.layer_norm_backward(r, x, x, r, weight=w, bias=b)
    assert g.x.shape == x.shape and g.weight.shape == (cols,)
    if rows == 0:
        assert not bool(g.weight.any()) and not bool(g.bias.any())


def test_the_same_call_gives_the_same_bits(tg):
    for rows, cols, pad in ((1000, 2048, 0), (333, 1001, 1), (200, 12000, 0)):
        x, kept, dy, dh = make(rows, cols, BF16, BF16, pad=pad)
        first = tg.layer_norm_backward(dy, dh, x, **kept)
        for _ in range(3):
            for a, b in zip(first, tg.layer_norm_backward(dy, dh, x, **kept)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(1, 520), (6, 521), (300, 4096)])
def test_plain_and_general_calls_agree(tg, rows, cols):
    """A call on a stream of its own, or with results given, takes another way through
    the binding: the same bits."""
    x, kept, dy, dh = make(rows, cols, BF16, F32)
    y, h = tg.layer_norm(x, **kept)
    other = tg.layer_norm(x, out=torch.empty_like(y), normed=torch.empty_like(h), **kept)
    assert torch.equal(y, other[0]) and torch.equal(h, other[1])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    calls = [lambda **k: tg.layer_norm(x, **kept, **k), lambda **k: tg.layer_norm_i8(x, **kept, **k),
             lambda **k: tg.quantize_rows(x, **k),
             lambda **k: tg.layer_norm_backward(dy, dh, x, **kept, **k)]
    for call in calls:
        a, b = call(), call(stream=stream)
        stream.synchronize()
        assert type(a) is type(b)
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert isinstance(a, tg.LayerNormGrads)
    weight = torch.nn.Parameter(kept["weight"])
    again = tg.layer_norm(x, **dict(kept, weight=weight))
    assert torch.equal(again[1], h) and not again[1].requires_grad


@pytest.mark.parametrize("cols", [777, 2048, 9000])
def test_two_captured_graphs_at_once(tg, cols):
    """Graphs captured one after the other on one stream share no workspace: replayed on two
    streams at the same time, each gives its own results."""
    cases = [make(400, cols, BF16, BF16, seed=s) for s in (1, 2)]
    want = [tg.layer_norm_backward(dy, dh, x, **kept) for x, kept, dy, dh in cases]
    graphs, got = [], []
    for x, kept, dy, dh in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(tg.layer_norm_backward(dy, dh, x, **kept))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_the_c_entry_with_a_workspace_of_the_library(tg):
    x, kept, dy, dh = make(64, 1000, F32, F32)
    want = tg.layer_norm_backward(dy, dh, x, **kept)
    out = [torch.empty_like(t) for t in (x, kept["residual"], kept["weight"], kept["bias"])]
    n = tg.tg_layer_norm_t(2, 2, 64, 1000, x.data_ptr(), x.stride(0), kept["residual"].data_ptr(),
                           kept["residual"].stride(0), kept["weight"].data_ptr(),
                           kept["bias"].data_ptr(), 1e-5)
    g = tg.tg_layer_norm_grad_t(dy.data_ptr(), dy.stride(0), dh.data_ptr(), dh.stride(0),
                                out[0].data_ptr(), out[0].stride(0), out[1].data_ptr(),
                                out[1].stride(0), out[2].data_ptr(), out[3].data_ptr(), None, 0)
    assert tg.tg_layer_norm_backward(n, g, torch.cuda.current_stream().cuda_stream) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_gradient_against_differences(tg):
    """The gradient's product with a direction, and the slope of the norm along it (64 bits)."""
    x, kept, dy, dh = make(9, 700, F32, F32)
    grads = tg.layer_norm_backward(dy, dh, x, **kept)
    inputs = [x, kept["residual"], kept["weight"], kept["bias"]]
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, (inp, grad) in enumerate(zip(inputs, grads)):
        way = torch.randn(inp.shape, generator=g, device="cuda").double()

        def total(step):
            moved = [t.double() + (step * way if j == i else 0) for j, t in enumerate(inputs)]
            r = ref.LayerNorm(moved[0], moved[1], weight=moved[2], bias=moved[3], eps=kept["eps"])
            return float((r.y * dy.double()).sum() + (r.h * dh.double()).sum())

        slope = (total(1e-5) - total(-1e-5)) / 2e-5
        along = float((grad.double() * way).sum())
        # fp32 gradients: 2^-24 of each term and the bounds' c; differences: 1e-10 of the curvature
        assert abs(slope - along) <= 1e-5 * float((grad.double() * way).abs().sum()), i


def test_refusals(tg):
    x, kept, dy, dh = make(4, 64, BF16, F32)
    with pytest.raises(TypeError):
        tg.layer_norm(x.int())
    with pytest.raises(TypeError):
        tg.layer_norm(x, kept["residual"].half())
    with pytest.raises(ValueError):
        tg.layer_norm(x, kept["residual"][:3])
    with pytest.raises(ValueError):
        tg.layer_norm(x, weight=kept["weight"].half())
    with pytest.raises(ValueError):
        tg.layer_norm(x, bias=kept["bias"][:5])
    with pytest.raises(ValueError):
        tg.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        tg.layer_norm(x.t())
    with pytest.raises(ValueError):
        tg.layer_norm(x, out=torch.empty_like(x))  # no residual, so no sum
    with pytest.raises(ValueError):
        tg.layer_norm_i8(x, out=torch.empty_like(x))
    with pytest.raises(TypeError):
        tg.layer_norm(x, kept["residual"], out=torch.empty_like(x))
    with pytest.raises(TypeError):
        tg.layer_norm_backward(dy.half(), dh, x, **kept)
    with pytest.raises(ValueError):
        tg.layer_norm_backward(dy, dh[:, :5], x, **kept)
    with pytest.raises(ValueError):
        tg.quantize_rows(torch.zeros(1, 131072, device="cuda"))


# ------------------------------------------------------------------ rows as codes

@pytest.mark.parametrize("dtype", [HALF, BF16, F32])
@pytest.mark.parametrize("cols", WIDTHS + [65536, 131071])
def test_codes(tg, dtype, cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    for rows, pad in ((5, 0), (3, 1)):
        x = (torch.randn(rows, cols + pad, generator=g, device="cuda") * 3).to(dtype)[:, :cols]
        codes, scale = tg.quantize_rows(x)
        want = ref.codes_of(x)
        assert codes.shape == x.shape and codes.dtype == torch.int8 and codes.stride(0) % 16 == 0
        assert torch.equal(scale, want[1]) and torch.equal(codes, want[0])


@pytest.mark.parametrize("dtype", [HALF, BF16, F32])
def test_codes_of_halves(tg, dtype):
    """Quotients that are halves go to the even code, at every code, and their neighbours
    to the nearer one."""
    for power in (0, -20, 3) + ((-140, 100) if dtype != HALF else ()):
        step = 2.0 ** power
        halves = torch.arange(-127, 127, device="cuda").double() + 0.5
        x = torch.cat((halves, torch.tensor([127.0], device="cuda").double())) * step
        near = torch.nextafter(x.float(), torch.full_like(x.float(), 1e38))
        for v in (x.float(), near, -near) if dtype == F32 else (x,):
            v = v.to(dtype)[None].contiguous()
            codes, scale = tg.quantize_rows(v)
            want = ref.codes_of(v)
            assert torch.equal(scale, want[1]) and torch.equal(codes, want[0])


def test_codes_of_small_and_large_rows(tg):
    rows = [torch.zeros(300), torch.full((300,), 65504.0), torch.full((300,), 3.4e38),
            torch.linspace(-1e-42, 1e-42, 300), torch.linspace(-1e-37, 1e-37, 300),
            torch.linspace(-3e38, 1e38, 300), torch.full((300,), 1e-45)]
    rows[0][7] = -0.0
    x = torch.stack(rows).cuda()
    # (the sixth row is not finite: its ends lie further apart than fp32 reaches)
    assert x.isfinite().all(dim=1).tolist() == [True] * 5 + [False, True]
    codes, scale = tg.quantize_rows(x)
    want = ref.codes_of(x)
    assert torch.equal(scale[:5], want[1][:5]) and bool(scale[5].isnan()) and torch.equal(scale[6:], want[1][6:])
    assert torch.equal(codes, want[0])
    x[1, 5], x[2, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    codes, scale = tg.quantize_rows(x)
    want = ref.codes_of(x)
    assert torch.equal(scale.isnan(), want[1].isnan()) and scale.isnan().nonzero().flatten().tolist() == [1, 2, 4, 5]
    assert torch.equal(codes, want[0])


@pytest.mark.parametrize("rows", [1, 150, 1000, 5000])
def test_codes_of_many_rows(tg, rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    for cols in (520, 4096):
        x = torch.randn(rows, cols, generator=g, device="cuda").to(BF16).clamp_(min=0)
        codes, scale = tg.quantize_rows(x)
        want = ref.codes_of(x)
        assert torch.equal(scale, want[1]) and torch.equal(codes, want[0])


def test_a_wait_for_another_block_that_runs_out_is_reported_once(tg):
    """Sums that are not sent: the gradient's kernel gives up within its limit and returns,
    the status says so once, and the next call is right."""
    x, kept, dy, dh = make(3, 20000, BF16, BF16)
    want = tg.layer_norm_backward(dy, dh, x, **kept)
    tg.sync_status()
    try:
        tg.tg_debug_set_wait_timeout_ns(20_000_000)
        tg.tg_debug_inject(1)
        tg.layer_norm_backward(dy, dh, x, **kept)
        with pytest.raises(tg.TgemmError) as e:
            tg.sync_status()
        assert e.value.status == tg.TG_ERR_TIMEOUT
        tg.sync_status()
    finally:
        tg.tg_debug_inject(0)
        tg.tg_debug_set_wait_timeout_ns(0)
    for a, b in zip(tg.layer_norm_backward(dy, dh, x, **kept), want):
        assert torch.equal(a, b)
    tg.sync_status()


@pytest.mark.parametrize("pad", [0, 1, 3])
def test_one_row_at_the_end_of_its_memory(tg, pad):
    """Matrices that begin and end where their allocation does (read off every boundary)."""
    for cols in (5, 517, 1031, 9001):
        for first in (0, 1):
            def place(kind):
                whole = torch.randn(3 * (cols + pad) - pad + first, device="cuda").to(kind)
                return torch.as_strided(whole, (3, cols), (cols + pad, 1), first)
            x, r, dy, dh = place(HALF), place(F32), place(F32), place(HALF)
            w = 1 + torch.randn(cols, device="cuda")
            want = ref.LayerNorm(x, r, weight=w, bias=w)
            want.check(*tg.layer_norm(x, r, weight=w, bias=w), f"{cols}")
            want.check_grads(tg.layer_norm_backward(dy, dh, x, r, weight=w, bias=w), dy, dh, f"{cols}")
