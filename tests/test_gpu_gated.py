"""GPU tests of the gated layer against plain implementations in 64 bits (bars as in
test_gpu_block_ops.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, DT, E, U, act_ref, act_slope_ref, close, make_weight, randn  # noqa: E402,F401

ACTS = ["silu", "gelu", "relu2", None, "gelu_tanh", "relu"]
SHAPES = [(1, 1, 1), (1, 2816, 768), (2, 768, 2816), (1, 8192, 4096), (3, 65, 7), (8, 2816, 768), (16, 100, 1000),
          (17, 300, 771), (33, 257, 129), (64, 768, 768), (100, 768, 2816), (129, 768, 256), (255, 511, 65), (256, 4000, 512),
          (300, 2815, 771), (1000, 768, 2816), (2048, 256, 768), (513, 1, 100), (700, 1000, 1), (1500, 3001, 320)]


def forward_check(x, wg, wu, act, dtype, y, g=None, u=None, what=""):
    xd, k = x.double(), x.shape[-1]
    rg, ru = xd @ wg.double().t(), xd @ wu.double().t()
    mg, mu = xd.abs() @ wg.double().abs().t(), xd.abs() @ wu.double().abs().t()
    c = 2 * (k / 16 + 4)
    # act(g) u: g's error times the slope (2 |g| or 1.2 at most) and u, u's times act(g), the
    # activation's own arithmetic about 8 roundings of its argument and value, one for the product
    value, slope = act_ref(rg, act), 2 * rg.abs() + 1.2 if act else torch.ones_like(rg)
    mag = (mg * slope + 8 * (rg.abs() + rg.square())) * ru.abs() + mu * value.abs()
    # (both factors' errors together: a second-order term, below one part in 2^10 of the first)
    close(y, value * ru, dtype, 1.01 * mag, c, ("y", what))
    if g is not None:
        close(g, rg, dtype, mg, c, ("g", what))
        close(u, ru, dtype, mu, c, ("u", what))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(A, shape, transposed, dtype):  # noqa: F811
    rows, n, k = shape
    for i, (act, keep, pad, off) in enumerate([("silu", False, 0, 0), ("gelu", True, 0, 0), ("relu2", True, 8, 0), (None, False, 1, 1),
                                               ("silu", True, 1, 0)]):
        x = randn(10 + i, rows, k, dtype=dtype, pad=pad, offset=off)
        wg, wu = make_weight(20 + i, n, k, dtype, transposed, pad, off), make_weight(30 + i, n, k, dtype, transposed, pad, off)
        got = A.gated_linear_forward(x, wg, wu, activation=act, save_preact=keep)
        forward_check(x, wg, wu, act, dtype, *(got if keep else (got,)), what=(act, pad, off))
    assert A.device_error() == A.OK


@pytest.mark.parametrize("act", ACTS, ids=str)
@pytest.mark.parametrize("rows", [1, 20, 400])
def test_activations(A, act, rows):  # noqa: F811
    x, wg, wu = randn(1, rows, 96, dtype="bf16"), make_weight(2, 300, 96, "bf16", False), make_weight(3, 300, 96, "bf16", False)
    y, g, u = A.gated_linear_forward(x, wg, wu, activation=act, save_preact=True)
    forward_check(x, wg, wu, act, "bf16", y, g, u)
    assert torch.equal(y, A.gated_linear_forward(x, wg, wu, activation=act))


def backward_check(dy, x, wg, wu, g, u, act, dtype, dw_type, got, parts=1, base=(None, None)):
    dx, dgate, dup = got
    rows, n, k = dy.shape[0], wg.shape[0], wg.shape[1]
    d, gd, ud, xd = dy.double(), g.double(), u.double(), x.double()
    value, slope = act_ref(gd, act), act_slope_ref(gd, act)
    dg, du = d * ud * slope, d * value
    # dg and du are rounded to the operands' type, once or in two parts; their own arithmetic: 16
    # roundings of slope and value and two products
    unit = U[dtype] if parts == 1 else U[dtype] ** 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    eg = unit * dg.abs() + 18 * E * d.abs() * ud.abs() * (2 * gd.abs() + 2) + tiny
    eu = unit * du.abs() + 18 * E * d.abs() * (gd.abs() + gd.square()) + tiny
    if dx is not None:
        c = 2 * (2 * parts * n / 16 + 4 * parts + 4)
        ref = dg @ wg.double() + du @ wu.double()
        mag = dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()
        close(dx, ref, dtype, mag + (eg @ wg.double().abs() + eu @ wu.double().abs()) / E / c, c, "dx")
    for got, z, ez, b, what in ((dgate, dg, eg, base[0], "dgate"), (dup, du, eu, base[1], "dup")):
        if got is None:
            continue
        c = 2 * 36 + parts * rows / 512 + 8 if dw_type == "f32" else 2 * (parts * rows / 16 + 8)
        ref, mag = z.t() @ xd, z.abs().t() @ xd.abs() + ez.t() @ xd.abs() / E / c
        if b is not None:
            ref, mag = ref + b.double(), mag + b.double().abs()
        close(got, ref, dw_type, mag, c, what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(5000, 256, 200), (9000, 64, 72)], ids=lambda s: "x".join(map(str, s)))
def test_backward(A, shape, transposed, dtype):  # noqa: F811
    rows, n, k = shape
    for i, (act, dw_type, pad, off, parts) in enumerate([("silu", "f32", 0, 0, 1), ("gelu", dtype, 0, 0, 2), ("relu2", "f32", 1, 1, 2),
                                                         (None, dtype, 8, 0, 1), ("silu", dtype, 1, 0, 1)]):
        dy, g, u = (randn(40 + 3 * i + j, rows, n, dtype=dtype, pad=pad, offset=off) for j in range(3))
        x = randn(70 + i, rows, k, dtype=dtype, pad=pad, offset=off)
        wg, wu = make_weight(80 + i, n, k, dtype, transposed, pad, off), make_weight(90 + i, n, k, dtype, transposed, pad, off)
        got = A.gated_linear_backward(dy, x, wg, wu, g, u, activation=act, dweight_dtype=DT[dw_type], dz_parts=parts)
        if n > 1 and k > 1:
            assert got[1].stride() == got[2].stride() == ((1, n) if transposed else (k, 1))
        backward_check(dy, x, wg, wu, g, u, act, dtype, dw_type, got, parts)
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dw_type", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", [(40, 96, 136), (3000, 300, 200), (4096, 2816, 768)], ids=lambda s: "x".join(map(str, s)))
def test_accumulate_and_subsets(A, shape, transposed, dw_type):  # noqa: F811
    """Added to what is there, into the two halves of one matrix; and one gradient without the other."""
    rows, n, k = shape
    dy, g, u = (randn(200 + j, rows, n, dtype="bf16") for j in range(3))
    x = randn(210, rows, k, dtype="bf16")
    both = randn(220, *((k, 2 * n) if transposed else (2 * n, k)), scale=k ** -0.5, dtype="bf16")
    both_grad = randn(230, *both.shape, dtype=dw_type)
    halves = (lambda t: (t[:, :n].t(), t[:, n:].t())) if transposed else (lambda t: (t[:n], t[n:]))  # noqa: E731
    (wg, wu), (dgate, dup) = halves(both), halves(both_grad)
    before = dgate.clone(), dup.clone()
    dx, a, b = A.gated_linear_backward(dy, x, wg, wu, g, u, dgate=dgate, dup=dup, accumulate=True)
    assert a.data_ptr() == dgate.data_ptr()
    backward_check(dy, x, wg, wu, g, u, "silu", "bf16", dw_type, (dx, a, b), base=before)
    only = A.gated_linear_backward(dy, x, wg, wu, g, u, need_dweight=False)
    assert only[1] is None and only[2] is None
    backward_check(dy, x, wg, wu, g, u, "silu", "bf16", dw_type, only)
    only = A.gated_linear_backward(dy, x, wg, wu, g, u, need_dx=False, dgate=dgate, dup=dup)
    assert only[0] is None
    backward_check(dy, x, wg, wu, g, u, "silu", "bf16", dw_type, only)
    forward_check(x, wg, wu, "silu", "bf16", A.gated_linear_forward(x, wg, wu))


def test_gradient_against_differences(A):  # noqa: F811
    """The operator's gradients against central differences of its own fp64 definition along random
    directions, at its rounded inputs: relative 2^-6 covers bf16's roundings of dg and du (2^-8 of the
    terms' root sum of squares, a sum of many) and the difference's own h^2 term."""
    rows, n, k, h = 60, 96, 80, 1e-4
    x, wg, wu = randn(1, rows, k, dtype="bf16"), make_weight(2, n, k, "bf16", False), make_weight(3, n, k, "bf16", False)
    dy = randn(4, rows, n, dtype="bf16")
    _, g, u = A.gated_linear_forward(x, wg, wu, save_preact=True)
    grads = A.gated_linear_backward(dy, x, wg, wu, g, u, dweight_dtype=torch.float32, dz_parts=2)
    point = [t.double() for t in (x, wg, wu)]
    value = lambda x, a, b: float((act_ref(x @ a.t(), "silu") * (x @ b.t()) * dy.double()).sum())  # noqa: E731
    for i in range(3):
        way = grads[i].double() / grads[i].double().norm()
        up, down = list(point), list(point)
        up[i], down[i] = point[i] + h * way, point[i] - h * way
        want = (value(*up) - value(*down)) / (2 * h)
        got = float((grads[i].double() * way).sum())
        assert abs(got - want) <= 2.0 ** -6 * abs(want), i


@pytest.mark.parametrize("rows", [1, 3, 300])
def test_infinities_and_nan_stay_in_their_rows(A, rows):  # noqa: F811
    x, wg, wu = randn(1, rows, 64, dtype="bf16"), make_weight(2, 96, 64, "bf16", False), make_weight(3, 96, 64, "bf16", False)
    clean = A.gated_linear_forward(x, wg, wu)
    x[rows // 2, 5] = float("nan")
    got = A.gated_linear_forward(x, wg, wu)
    assert torch.isnan(got[rows // 2]).all()
    keep = torch.arange(rows, device="cuda") != rows // 2
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("rows", [1, 2, 40, 500])
@pytest.mark.parametrize("n", [95, 96, 2815])
def test_nothing_beside_the_results(A, rows, n):  # noqa: F811
    """Results in wider buffers: what is beside them stays, NaN beside the operands stays out."""
    def wide(shape, fill):
        t = torch.full((shape[0] + 2, shape[1] + 24), fill, device="cuda", dtype=torch.bfloat16)
        return t, t[1:-1, 8:8 + shape[1]]
    _, x = wide((rows, 72), float("nan"))
    x.copy_(randn(1, rows, 72, dtype="bf16"))
    weights = []
    for s in (2, 3):
        w = wide((n, 72), float("nan"))[1]
        w.copy_(make_weight(s, n, 72, "bf16", False))
        weights.append(w)
    full, out = wide((rows, n), 7.0)
    y = A.gated_linear_forward(x, *weights, out=out)
    assert y.data_ptr() == out.data_ptr()
    forward_check(x, *weights, "silu", "bf16", out)
    out.fill_(7.0)
    assert (full == 7.0).all()


def test_empty(A):  # noqa: F811
    x, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), make_weight(2, 96, 64, "bf16", False)
    y, g, u = A.gated_linear_forward(x, w, w, save_preact=True)
    assert y.shape == g.shape == u.shape == (0, 96)
    dx, dg, du = A.gated_linear_backward(y, x, w, w, g, u)
    assert dx.shape == (0, 64) and not dg.any() and not du.any()


def test_graph_and_streams(A):  # noqa: F811
    """Captured and replayed with new inputs, and on another stream: the same bits as a plain call."""
    rows, n, k = 700, 520, 264
    x, wg, wu = randn(1, rows, k, dtype="bf16"), make_weight(2, n, k, "bf16", False), make_weight(3, n, k, "bf16", False)
    dy = randn(4, rows, n, dtype="bf16")

    def both():
        y, g, u = A.gated_linear_forward(x, wg, wu, save_preact=True)
        return (y, g, u) + A.gated_linear_backward(dy, x, wg, wu, g, u, dweight_dtype=torch.float32)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(randn(5, rows, k, dtype="bf16"))
    graph.replay()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = A.gated_linear_forward(x, wg, wu, stream=s)
    s.synchronize()
    assert torch.equal(other, want[0])


def test_past_32_bit_offsets(A):  # noqa: F811
    """Rows whose elements lie past 2^31 in x, in y and in the kept factors."""
    rows, n, k = (1 << 25) + 5, 64, 72
    x = torch.zeros(rows, k, device="cuda", dtype=torch.bfloat16)
    tail = randn(1, 300, k, dtype="bf16")
    x[-300:] = tail
    wg, wu = make_weight(2, n, k, "bf16", False), make_weight(3, n, k, "bf16", False)
    y, g, u = A.gated_linear_forward(x, wg, wu, save_preact=True)
    forward_check(tail, wg, wu, "silu", "bf16", y[-300:], g[-300:], u[-300:])
    assert not y[:-300].any()
    dy = torch.zeros_like(y)
    dy[-300:] = randn(4, 300, n, dtype="bf16")
    got = A.gated_linear_backward(dy, x, wg, wu, g, u)
    small = A.gated_linear_backward(dy[-300:], tail, wg, wu, g[-300:], u[-300:], dweight_dtype=torch.float32)
    assert not got[0][:-300].any()
    backward_check(dy[-300:], tail, wg, wu, g[-300:], u[-300:], "silu", "bf16", "bf16", (got[0][-300:], got[1], got[2]))
    assert small[0].shape == (300, k)
