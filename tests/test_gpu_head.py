"""GPU tests of the head's cross entropy against plain implementations in 64 bits (bars as in
test_gpu_block_ops.py)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, DT, E, U, close, make_weight, randn  # noqa: E402,F401

SHAPES = [(1, 1, 1), (1, 50304, 768), (7, 700, 5000), (1, 1001, 5001), (4, 50257, 771), (3, 33, 4000), (2, 131072, 64), (4, 16, 4096), (30, 16384, 1024), (100, 50304, 200), (250, 257, 300), (2, 7, 5), (3, 65, 64), (5, 1000, 100), (17, 50257, 130), (64, 4096, 768), (129, 300, 771),
          (257, 511, 256), (300, 50304, 64), (777, 5003, 771), (1500, 256, 96), (2048, 8192, 520)]


def make_targets(seed, rows, vocab, wide=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if rows > 4:
        t[::5] = -1
        t[1], t[2] = 0, vocab - 1
    return t if wide else t.int()


def logits(x, w):
    """z and the error that the products may leave: 2 E per 16-deep step of the magnitudes."""
    k = x.shape[-1]
    return x.double() @ w.double().t(), 2 * (k / 16 + 4) * E * (x.double().abs() @ w.double().abs().t())


def forward_check(x, w, t, loss, lse, what=""):
    z, ez = logits(x, w)
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    # the exponentials 4 E each (2^-22) and one rounding of an exponent that counts; sums in chains of 8,
    # then the parts of 64 columns in eight shares at least, each step a sum and two factors of 5 E; the
    # logarithm and its sum
    parts = math.ceil(w.shape[0] / 256) * 4
    bar = (p * ez).sum(1) + E * (4 + 2 + 24 + 11 * (parts / 8 + 9) + 4 * want.abs() + 4)
    # (where one logit's error shifts it by d, lse moves by p d (1 + d) at most)
    assert ((lse.double() - want).abs() <= 1.01 * bar).all(), (what, float(((lse.double() - want).abs() / bar).max()))
    if t is None:
        assert loss is None
        return
    live = t >= 0
    at = t.clamp_min(0).long()[:, None]
    ref = torch.where(live, want - z.gather(1, at)[:, 0], torch.zeros_like(want))
    bar = bar + ez.gather(1, at)[:, 0] + 2 * E * ref.abs()
    assert ((loss.double() - ref).abs() <= 1.01 * bar).all(), (what, float(((loss.double() - ref).abs() / bar).max()))
    assert (loss[~live] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(A, shape, transposed, dtype):  # noqa: F811
    rows, vocab, k = shape
    for i, (scale, pad, off, wide) in enumerate([(1.0, 0, 0, True), (6.0, 8, 0, False), (2.0, 1, 1, True)]):
        x = randn(10 + i, rows, k, scale=scale, dtype=dtype, pad=pad, offset=off)
        w, t = make_weight(20 + i, vocab, k, dtype, transposed, pad, off), make_targets(30 + i, rows, vocab, wide)
        loss, lse = A.linear_cross_entropy(x, w, t)
        forward_check(x, w, t, loss, lse, (scale, pad, off))
        none, again = A.linear_cross_entropy(x, w)
        assert none is None and torch.equal(again, lse)
    assert A.device_error() == A.OK


def backward_check(x, w, t, lse, gl, dtype, dw_type, got, base=None):
    z, ez = logits(x, w)
    live = t >= 0
    g = torch.where(live, gl.double(), torch.zeros_like(gl.double()))[:, None]
    p = torch.exp(z - lse.double()[:, None])
    d = g * p
    hot = torch.arange(t.numel(), device="cuda")[live]
    d[hot, t[live].long()] -= g[hot, 0]
    # p: the logit's error, the exponent's (|z| and |lse| with log2(e) rounded, one product and one sum:
    # 2 E of them together), 4 E of the exponential; d: two roundings, three of the factor that it is
    # taken over (1 / it, g times that, the results times it), and its own to the operands' type
    ep = p * (ez + 3 * E * (z.abs() + lse.double().abs()[:, None]) + 8 * E)
    ed = g.abs() * ep * 1.01 + (5 * E + U[dtype]) * d.abs()
    if dtype == "f16":  # below fp16's smallest normal value over the largest |g|'s 2^13
        ed = ed + 2.0 ** -25 * 2.0 ** -13 * float(g.abs().max()) * (g != 0)
    dx, dw = got
    rows, vocab, k = x.shape[0], w.shape[0], w.shape[1]
    if dx is not None:
        c = 2 * (vocab / 16 + 8)
        close(dx, d @ w.double(), dtype, d.abs() @ w.double().abs() + ed @ w.double().abs() / E / c, c, "dx")
    if dw is not None:
        c = 2 * 36 + rows / 512 + 8 if dw_type == "f32" else 2 * (rows / 16 + 8)
        ref, mag = d.t() @ x.double(), d.abs().t() @ x.double().abs() + ed.t() @ x.double().abs() / E / c
        if base is not None:
            ref, mag = ref + base.double(), mag + base.double().abs()
        close(dw, ref, dw_type, mag, c, "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(A, shape, transposed, dtype):  # noqa: F811
    rows, vocab, k = shape
    for i, (dw_type, pad, off, size) in enumerate([(dtype, 0, 0, 1.0 / rows), ("f32", 8, 0, 1.0), (dtype, 1, 1, 1e-4)]):
        x = randn(40 + i, rows, k, scale=2.0, dtype=dtype, pad=pad, offset=off)
        w, t = make_weight(50 + i, vocab, k, dtype, transposed, pad, off), make_targets(60 + i, rows, vocab, i == 0)
        gl = randn(70 + i, rows, scale=size)
        _, lse = A.linear_cross_entropy(x, w, t)
        got = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=DT[dw_type])
        if vocab > 1 and k > 1:
            assert got[1].stride() == ((1, vocab) if transposed else (k, 1))
        backward_check(x, w, t, lse, gl, dtype, dw_type, got)
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_pieces(A, transposed, dtype):  # noqa: F811
    """More logits than a piece takes: three pieces, the last one narrow and odd."""
    rows, vocab, k = 20000, 13001, 72
    x, w = randn(1, rows, k, scale=2.0, dtype=dtype), make_weight(2, vocab, k, dtype, transposed)
    t, gl = make_targets(3, rows, vocab), randn(4, rows, scale=1.0 / rows)
    loss, lse = A.linear_cross_entropy(x, w, t)
    forward_check(x, w, t, loss, lse)
    got = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=torch.float32)
    backward_check(x, w, t, lse, gl, dtype, "f32", got)
    only, none = A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dweight=False)
    assert none is None
    backward_check(x, w, t, lse, gl, dtype, dtype, (only, None))
    none, only = A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dx=False)
    assert none is None
    backward_check(x, w, t, lse, gl, dtype, dtype, (None, only))


@pytest.mark.parametrize("dw_type", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_accumulate(A, transposed, dw_type):  # noqa: F811
    rows, vocab, k = 600, 1003, 136
    x, w = randn(1, rows, k, dtype="bf16"), make_weight(2, vocab, k, "bf16", transposed)
    t, gl = make_targets(3, rows, vocab), randn(4, rows)
    _, lse = A.linear_cross_entropy(x, w, t)
    dw = randn(5, *((k, vocab) if transposed else (vocab, k)), dtype=dw_type)
    dw = dw.t() if transposed else dw
    base = dw.clone()
    got = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight=dw, accumulate=True)
    assert got[1].data_ptr() == dw.data_ptr()
    backward_check(x, w, t, lse, gl, "bf16", dw_type, got, base)


def test_gradient_against_differences(A):  # noqa: F811
    """The gradients against central differences of the definition in 64 bits along their own
    directions; 2^-6 covers bf16's rounding of d (2^-8 of each of many terms) and the differences' h^2."""
    rows, vocab, k, h = 90, 300, 80, 1e-4
    x, w, t = randn(1, rows, k, dtype="bf16"), make_weight(2, vocab, k, "bf16", False), make_targets(3, rows, vocab)
    gl = randn(4, rows).abs()
    _, lse = A.linear_cross_entropy(x, w, t)
    grads = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=torch.float32)
    live = (t >= 0).double() * gl.double()
    value = lambda x, w: float((torch.nn.functional.cross_entropy(x @ w.t(), t.clamp_min(0), reduction="none") * live).sum())  # noqa: E731
    point = [x.double(), w.double()]
    for i in range(2):
        way = grads[i].double() / grads[i].double().norm()
        up, down = list(point), list(point)
        up[i], down[i] = point[i] + h * way, point[i] - h * way
        want, got = (value(*up) - value(*down)) / (2 * h), float((grads[i].double() * way).sum())
        assert abs(got - want) <= 2.0 ** -6 * abs(want), i


def test_tokens_that_cannot_be(A):  # noqa: F811
    """Logits of -inf: left out; a row of nothing else; NaN and +inf rows; targets beyond the vocabulary."""
    rows, vocab, k = 300, 1000, 64
    x, w = randn(1, rows, k, dtype="bf16"), make_weight(2, vocab, k, "bf16", False)
    x[:, 0] = 1.0
    w[::3, 0] = -math.inf
    t = make_targets(3, rows, vocab)
    t[7], t[8], t[9] = 3, vocab, 1 << 40
    x[20, 5], x[21, 0] = math.nan, -1.0  # row 21: +inf where the others have -inf
    loss, lse = A.linear_cross_entropy(x, w, t)
    z = torch.where(torch.isinf(w[:, :1].t()), -math.inf, (x.double() @ w.double().nan_to_num(neginf=0.0).t()))
    want = torch.logsumexp(z, 1)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[20:22] = False
    assert ((lse.double() - want)[keep].abs() < 1e-3).all() and torch.isnan(lse[20:22]).all()
    assert math.isinf(float(loss[7])) and torch.isnan(loss[8:10]).all()
    live = keep & (t >= 0) & (t < vocab) & (t % 3 != 0)
    ref = want - z.gather(1, t.clamp(0, vocab - 1)[:, None])[:, 0]
    assert ((loss.double() - ref)[live].abs() < 1e-3).all()
    # the gradient of a weight row that cannot be is 0, and of one beyond the vocabulary p alone
    gl = torch.ones(rows, device="cuda")
    gl[20:22] = 0.0
    _, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dx=False, dweight_dtype=torch.float32)
    hit = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    hit[t[(t >= 0) & (t < vocab)]] = True
    # (x's own NaN, in column 5 of row 20, reaches that column through the product: 0 NaN is NaN)
    others = torch.arange(k, device="cuda") != 5
    assert torch.isnan(dw[:, 5]).all() and not torch.isnan(dw[:, others]).any()
    assert not dw[(torch.arange(vocab, device="cuda") % 3 == 0) & ~hit][:, others].any()
    w[:, 0] = -math.inf
    x[21, 0] = 1.0
    loss, lse = A.linear_cross_entropy(x, w, t)
    rest = torch.arange(rows, device="cuda") != 20
    assert (lse[rest] == -math.inf).all() and (loss[rest & (t >= 0) & (t < vocab)] == math.inf).all() and (loss[t < 0] == 0).all()
    _, dw = A.linear_cross_entropy_backward(x, w, t, lse, torch.where(rest, 1.0, 0.0), need_dx=False)
    assert not dw[:, others].any()


def test_large_logits(A):  # noqa: F811
    """Logits in the thousands, where an exponential without the maximum would overflow, and equal ones."""
    x = torch.zeros(40, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(700, 64, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 64.0
    w[:, 0] = 64.0
    w[::2, 0] = -64.0
    t = torch.arange(40, device="cuda")
    loss, lse = A.linear_cross_entropy(x, w, t)
    want = 4096.0 + math.log(350.0)
    assert (lse - want).abs().max() <= want * 4 * E
    assert torch.equal(loss, lse - torch.where(t % 2 == 0, -4096.0, 4096.0))


@pytest.mark.parametrize("rows", [1, 2, 5, 40, 200, 300, 900])
@pytest.mark.parametrize("transposed", [False, True])
def test_low_logits(A, transposed, rows):  # noqa: F811
    """Logits far below 0 only, where 2 to the power of their distance from 0 overflows; the same behind columns of -inf."""
    vocab, k = 700, 64
    x = torch.zeros(rows, k, device="cuda", dtype=torch.bfloat16)
    w = make_weight(1, vocab, k, "bf16", transposed)
    w.zero_()
    x[:, 0], x[:, 1] = 64.0, 1.0
    w[:, 0] = torch.where(torch.arange(vocab, device="cuda") % 256 < 128, -64.0, -4.0).bfloat16()
    w[:, 1] = torch.arange(vocab, device="cuda").remainder(5).bfloat16()
    t = make_targets(2, rows, vocab)
    for least in (0, 40):
        w[:least, 0] = -math.inf
        loss, lse = A.linear_cross_entropy(x, w, t)
        z = x.double() @ w.double().nan_to_num(neginf=0.0).t()  # (exact in fp32 as well)
        z[:, :least] = -math.inf
        want = torch.logsumexp(z, 1)
        # forward_check's without the products' part
        parts = math.ceil(vocab / 256) * 4
        bar = E * (34 + 11 * (parts / 8 + 9) + 4 * want.abs())
        assert ((lse.double() - want).abs() <= 1.01 * bar).all()
        ref = want - z.gather(1, t.clamp_min(0)[:, None])[:, 0]
        live = (t >= 0) & ~torch.isinf(ref)
        assert ((loss.double() - ref).abs() <= 1.01 * (bar + 2 * E * ref.abs()))[live].all()
        assert (loss[t < 0] == 0).all() and (loss[(t >= 0) & torch.isinf(ref)] == math.inf).all()


def test_rows_past_the_last_and_workspace(A):  # noqa: F811
    """The caller's workspace, and nothing written beside a gradient given in wider rows."""
    rows, vocab, k = 130, 515, 77
    x, w, t, gl = randn(1, rows, k, dtype="bf16"), make_weight(2, vocab, k, "bf16", False), make_targets(3, rows, vocab), randn(4, rows)
    ws = torch.empty(1 << 24, device="cuda", dtype=torch.uint8)
    loss, lse = A.linear_cross_entropy(x, w, t, workspace=ws)
    forward_check(x, w, t, loss, lse)
    full = torch.full((vocab + 2, k + 19), 7.0, device="cuda")
    dw = full[1:-1, 8:8 + k]
    backward_check(x, w, t, lse, gl, "bf16", "f32", A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight=dw, workspace=ws))
    dw.fill_(7.0)
    assert (full == 7.0).all()
    with pytest.raises(A.AnvilError, match="WORKSPACE"):
        A.linear_cross_entropy(x, w, t, workspace=ws[:256])


def test_refusals(A):  # noqa: F811
    x, w, t, f = randn(1, 4, 8, dtype="bf16"), make_weight(2, 60, 8, "bf16", False), make_targets(3, 4, 60), randn(4, 4)
    with pytest.raises(ValueError, match="dweight must have weight's shape and order"):
        A.linear_cross_entropy_backward(x, w, t, f, f, dweight=make_weight(2, 60, 8, "bf16", True))
    with pytest.raises(ValueError, match="current CUDA device"):
        A.linear_cross_entropy(x, w.cpu(), t)
    with pytest.raises(A.AnvilError, match="ALIAS"):
        A.linear_cross_entropy_backward(x, w, t, f, f, dweight=w)


def test_empty(A):  # noqa: F811
    x, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), make_weight(2, 96, 64, "bf16", False)
    t = torch.empty(0, device="cuda", dtype=torch.int64)
    loss, lse = A.linear_cross_entropy(x, w, t)
    assert loss.shape == lse.shape == (0,)
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, loss)
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_graph_and_streams(A, dtype):  # noqa: F811
    rows, vocab, k = 700, 5000, 264
    x, w, t = randn(1, rows, k, dtype=dtype), make_weight(2, vocab, k, dtype, False), make_targets(3, rows, vocab)
    gl = randn(4, rows)

    def both():
        loss, lse = A.linear_cross_entropy(x, w, t)
        return (loss, lse) + A.linear_cross_entropy_backward(x, w, t, lse, gl)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(randn(5, rows, k, dtype=dtype))
    t.copy_(make_targets(6, rows, vocab))
    graph.replay()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = A.linear_cross_entropy(x, w, t, stream=s)
    s.synchronize()
    assert torch.equal(other[0], want[0])


def test_past_32_bit_offsets(A):  # noqa: F811
    """A weight of more than 2^31 elements, and rows of x beyond them."""
    vocab, k = (1 << 21) + 77, 1032
    w = torch.zeros(vocab, k, device="cuda", dtype=torch.bfloat16)
    w[-500:] = make_weight(1, 500, k, "bf16", False)
    x = randn(2, 40, k, dtype="bf16")
    t = torch.arange(vocab - 40, vocab, device="cuda")
    loss, lse = A.linear_cross_entropy(x, w, t)
    z = x.double() @ w[-500:].double().t()
    want = torch.logsumexp(torch.cat([z, math.log(vocab - 500) * torch.ones(40, 1, device="cuda").double()], 1), 1)
    assert (lse.double() - want).abs().max() < 1e-4
    assert (loss.double() - (want - z.gather(1, (t - (vocab - 500))[:, None])[:, 0])).abs().max() < 1e-4
    gl = randn(3, 40)
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl)
    d = torch.exp(z - lse.double()[:, None])
    d[torch.arange(40), t - (vocab - 500)] -= 1.0
    d = d * gl.double()[:, None]
    # d's rounding to bf16 (2^-8) and the results' own, relative to the sums of magnitudes
    assert ((dw[-500:].double() - d.t() @ x.double()).abs() <= 2.0 ** -7 * (d.abs().t() @ x.double().abs())).all()
    assert ((dx.double() - d @ w[-500:].double()).abs() <= 2.0 ** -7 * (d.abs() @ w[-500:].double().abs()) + 1e-6).all()
