"""GPU tests of the operators around the banks (layer norm, the linear layer, token log
probabilities) against plain implementations in 64 bits on the same inputs.

Bars.  U is the unit roundoff of the result's type, half the spacing of its values just above
a power of two (bf16 has 8 significant bits: 2^-8; fp16 11: 2^-11; for fp32 two roundings,
2^-23), E = 2^-24 that of fp32.  A result may be off by U |ref| for its own rounding, plus the fp32
arithmetic behind it: C E times the sum of the magnitudes that were added, where C counts
the roundings along one chain (derived beside each bar).  Products of 16-bit operands on the
tensor cores are exact, their sums truncate: 2 E per 16-deep step of the sum of magnitudes.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -23}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from polynomial_matrix_whitening_gb300 import anvil
    return anvil


def randn(seed, *shape, scale=1.0, dtype="f32", pad=0, offset=0):
    """Seeded normal values; pad: a view of rows that are `pad` wider; offset: the view
    starts that many elements into its rows (unaligned)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = shape[:-1] + (shape[-1] + pad + offset,)
    t = (torch.randn(full, generator=g, device="cuda") * scale).to(DT[dtype])
    return t[..., offset:offset + shape[-1]]


def close(got, ref, dtype, magnitude, c, what):
    """Every element within U |ref| + c E magnitude (fp16's subnormals: 2^-24 absolute)."""
    bar = U[dtype] * ref.abs() + c * E * magnitude + (2.0 ** -24 if dtype == "f16" else 1e-37)
    bad = (got.double() - ref).abs() > bar
    assert not torch.isnan(got).any(), what
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / bar).max()))


# ---------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (1, 768), (3, 7), (5, 64), (33, 65), (37, 256), (300, 768), (9, 1023), (17, 1024),
               (41, 2816), (7, 3000), (5, 4096), (3, 5001), (4, 8192), (2, 10000), (2, 16384), (2, 16383), (2000, 96)]


def norm_ref(x, w, b, eps):
    x = x.double()
    mu = x.mean(-1, keepdim=True)
    c = x - mu
    rs = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
    return c * rs * w.double() + b.double(), mu[..., 0], rs[..., 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_forward(A, shape, dtype):
    rows, n = shape
    for k, (pad, off, wt) in enumerate([(0, 0, "f32"), (1, 0, dtype), (8, 1, "f32")]):
        x = randn(100 + k, rows, n, scale=2.0, dtype=dtype, pad=pad, offset=off)
        w, b = 1 + randn(200 + k, n, scale=0.2), randn(300 + k, n, scale=0.2)
        w, b = w.to(DT[wt]), b.to(DT[wt])
        y, mean, rstd = A.layernorm_forward(x, w, b, 1e-5)
        ry, rm, rr = norm_ref(x, w, b, 1e-5)
        size = x.double().abs().amax(-1)
        # a sum's chain: at most 32 terms in a thread, 5 + 4 shuffles and warps, a division
        close(mean, rm, "f32", size, 48, "mean")
        # (x - mean)^2 doubles the mean's error; rstd has half the variance's relative error
        # (eps holds it where the variance is small)
        close(rstd, rr, "f32", rr * (1 + (size * rr).square()), 128, "rstd")
        h = (ry - b.double()).abs()
        close(y, ry, dtype, (h + b.double().abs()) * (1 + (size * rr).square())[:, None]
              + (size * rr)[:, None] * w.double().abs(), 192, "y")
    assert A.device_error() == A.OK


def norm_grad_ref(dy, x, mean, rstd, w, res):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy * (w.double() if w is not None else 1.0)
    m1, m2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - m1 - h * m2)
    mag = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True))
    if res is not None:
        dx, mag = dx + res.double(), mag + res.double().abs()
    return dx, (dy * h).sum(0), dy.sum(0), mag, (dy * h).abs().sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_backward(A, shape, dtype):
    rows, n = shape
    for k, (pad, off, wt, with_res) in enumerate([(0, 0, "f32", False), (1, 0, dtype, True), (8, 1, "f32", True)]):
        x = randn(400 + k, rows, n, scale=2.0, dtype=dtype, pad=pad, offset=off)
        dy = randn(500 + k, rows, n, dtype=dtype, pad=pad)
        res = randn(600 + k, rows, n, dtype=dtype, pad=off) if with_res else None
        w = (1 + randn(700 + k, n, scale=0.2)).to(DT[wt])
        _, mean, rstd = A.layernorm_forward(x, w, w, 1e-5)
        dx, dw, db = A.layernorm_backward(dy, x, mean, rstd, w, residual_grad=res)
        rx, rw, rb, mx, mw, mb = norm_grad_ref(dy, x, mean, rstd, w, res)
        h_err = (x.double().abs().amax(1) * rstd.double())[:, None]  # x - mean rounds relative to |x|
        close(dx, rx, dtype, mx * (1 + h_err), 128, "dx")
        # rows per block and partial sums per column: at most 2000 rows here, in chains of
        # at most 64 + 16 + 40 terms
        close(dw, rw, "f32", mw * (1 + float(h_err.max())) + 1e-30, 128, "dweight")
        close(db, rb, "f32", mb, 128, "dbias")
    assert A.device_error() == A.OK


# Enough rows for the kernels that keep several rows on their way, with rows left over that do
# not fill every team's share, for each width of a team; and rows off the 16-byte boundaries.
NORM_MANY = [(117003, 512), (58501, 1000), (29301, 2000), (14701, 2816), (14651, 4000), (7403, 8000),
             (29501, 300), (14801, 1023), (3701, 1500), (1901, 2815), (1003, 5001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("shape", NORM_MANY, ids=lambda s: "x".join(map(str, s)))
def test_norm_many_rows(A, shape, pad, dtype):
    rows, n = shape
    with_res = (rows + pad) % 2 == 0
    x = randn(110, rows, n, scale=2.0, dtype=dtype, pad=pad)
    dy = randn(111, rows, n, dtype=dtype, pad=pad)
    res = randn(112, rows, n, dtype=dtype, pad=pad) if with_res else None
    w, b = 1 + randn(113, n, scale=0.2), randn(114, n, scale=0.2)
    y, mean, rstd = A.layernorm_forward(x, w, b, 1e-5)
    ry, rm, rr = norm_ref(x, w, b, 1e-5)
    size = x.double().abs().amax(-1)
    close(mean, rm, "f32", size, 48, "mean")
    close(rstd, rr, "f32", rr * (1 + (size * rr).square()), 128, "rstd")
    close(y, ry, dtype, ((ry - b.double()).abs() + b.double().abs()) * (1 + (size * rr).square())[:, None]
          + (size * rr)[:, None] * w.double().abs(), 192, "y")
    del y, ry
    dx, dw, db = A.layernorm_backward(dy, x, mean, rstd, w, residual_grad=res)
    rx, rw, rb, mx, mw, mb = norm_grad_ref(dy, x, mean, rstd, w, res)
    h_err = (x.double().abs().amax(1) * rstd.double())[:, None]
    close(dx, rx, dtype, mx * (1 + h_err), 128, "dx")
    # a column's chain: at most 117003 / (152 * 2 * 8) rows a team, 8 teams, 304 blocks by 16, 16
    c = 2 * (rows // 152 // 2 + 1 if n > 512 else 49) + 8 + 19 + 16 + 16
    close(dw, rw, "f32", mw * (1 + float(h_err.max())) + 1e-30, c, "dweight")
    close(db, rb, "f32", mb, c, "dbias")
    # in place, and without what was not asked for: the same bits
    again = A.layernorm_backward(dy, x, mean, rstd, w, residual_grad=res, weight_grads=False, out=dy)
    assert torch.equal(again[0], dx) and again[1] is None
    assert A.device_error() == A.OK


def test_norm_in_place_and_no_affine(A):
    x = randn(1, 130, 768, dtype="bf16")
    y, mean, rstd = A.layernorm_forward(x)
    one, zero = torch.ones(768, device="cuda"), torch.zeros(768, device="cuda")
    y2, _, _ = A.layernorm_forward(x, one, zero)
    assert torch.equal(y, y2)
    dy, res = randn(2, 130, 768, dtype="bf16"), randn(3, 130, 768, dtype="bf16")
    want = A.layernorm_backward(dy, x, mean, rstd, residual_grad=res)
    for target in ("dy", "x", "res"):
        t = dict(dy=dy.clone(), x=x.clone(), res=res.clone())
        got = A.layernorm_backward(t["dy"], t["x"], mean, rstd, residual_grad=t["res"], out=t[target])
        assert got[0].data_ptr() == t[target].data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), target
    xi = x.clone()
    assert torch.equal(A.layernorm_forward(xi, out=xi)[0], y)
    only = A.layernorm_backward(dy, x, mean, rstd, residual_grad=res, weight_grads=False)
    assert torch.equal(only[0], want[0]) and only[1] is None


def test_norm_constant_and_nan_rows(A):
    x = randn(4, 6, 768, dtype="f32")
    x[1] = 3.5          # no variance: rstd = eps^-1/2, y = bias
    x[3, 5] = math.nan  # stays in its row
    b = randn(5, 768)
    y, mean, rstd = A.layernorm_forward(x, None, b, 1e-5)
    assert float(mean[1]) == 3.5 and abs(float(rstd[1]) * math.sqrt(1e-5) - 1) < 1e-6
    assert torch.equal(y[1], b)
    assert torch.isnan(y[3]).all() and not torch.isnan(y[[0, 1, 2, 4, 5]]).any()


def test_norm_gradient_against_differences(A):
    """The directional derivative of the plain forward in 64 bits (central differences)."""
    x, w, b = randn(6, 5, 257), 1 + randn(7, 257, scale=0.2), randn(8, 257, scale=0.2)
    dy = randn(9, 5, 257)
    _, mean, rstd = A.layernorm_forward(x, w, b)
    dx, dw, db = A.layernorm_backward(dy, x, mean, rstd, w)
    h = 1e-5

    def loss(dxs, dws, dbs):
        return (norm_ref(x.double() + dxs, w.double() + dws, b.double() + dbs, 1e-5)[0] * dy.double()).sum()
    zero = 0.0
    for g, k, shape in ((dx, 0, (5, 257)), (dw, 1, (257,)), (db, 2, (257,))):
        v = randn(20 + k, *shape).double()
        arg = [[zero] * 3, [zero] * 3]
        arg[0][k], arg[1][k] = h * v, -h * v
        num = (loss(*arg[0]) - loss(*arg[1])) / (2 * h)
        # the difference's own error is O(h^2) and 1e-16/h; the gradient's about 1e-6 of its terms
        assert abs(float((g.double() * v).sum() - num)) < 1e-4 * float((g.double() * v).abs().sum())


def test_norm_empty(A):
    x = torch.empty((0, 768), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = A.layernorm_forward(x)
    assert y.shape == (0, 768) and mean.shape == (0,)
    dx, dw, db = A.layernorm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 768) and not dw.any() and not db.any()


# ---------------------------------------------------------------- the linear layer
def act_ref(z, kind):
    if kind in (None, "none"):
        return z
    if kind == "relu":
        return z.clamp_min(0)
    if kind == "relu2":
        return z.clamp_min(0).square()
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_slope_ref(z, kind):
    z = z.detach().clone().requires_grad_(True)
    act_ref(z, kind).sum().backward()
    return z.grad


LINEAR_SHAPES = [(1, 1, 1), (1, 768, 2816), (1, 2816, 768), (3, 65, 7), (8, 2816, 768), (16, 100, 1000), (17, 300, 771),
                 (33, 257, 129), (64, 768, 768), (100, 768, 2816), (128, 130, 64), (129, 768, 256), (255, 511, 65),
                 (300, 2815, 771), (1000, 768, 2816), (2048, 256, 768), (513, 1, 100), (700, 1000, 1)]


def make_weight(seed, n, k, dtype, transposed, pad=0, offset=0):
    shape = (k, n) if transposed else (n, k)
    w = randn(seed, *shape, scale=k ** -0.5, dtype=dtype, pad=pad, offset=offset)
    return w.t() if transposed else w


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", LINEAR_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_linear_forward(A, shape, transposed, dtype):
    rows, n, k = shape
    for i, (act, bias, res, z, pad, off) in enumerate([(None, None, False, False, 0, 0), ("relu2", "f32", False, True, 0, 0),
                                                       ("gelu", dtype, True, True, 8, 0), ("silu", dtype, True, False, 1, 1)]):
        x = randn(800 + i, rows, k, dtype=dtype, pad=pad, offset=off)
        w = make_weight(900 + i, n, k, dtype, transposed, pad, off)
        b = randn(1000 + i, n, scale=0.3).to(DT[bias]) if bias else None
        r = randn(1100 + i, rows, n, dtype=dtype, pad=pad) if res else None
        got = A.linear_forward(x, w, b, activation=act, residual=r, save_preact=z)
        y = got[0] if z else got
        zr = x.double() @ w.double().t()
        mag = x.double().abs() @ w.double().abs().t()
        if b is not None:
            zr, mag = zr + b.double(), mag + b.double().abs()
        yr = act_ref(zr, act)
        # the accumulator: 2 E per 16-deep step; an activation's slope is at most 2 |z| (relu2)
        # or 1.2, its own arithmetic about 8 roundings of its argument and value
        c = 2 * (k / 16 + 4)
        slope = 2 * zr.abs() + 1.2 if act else torch.ones_like(zr)
        ymag = mag * slope + (8 * (zr.abs() + zr.square()) if act else 0)
        if r is not None:
            yr, ymag = yr + r.double(), ymag + r.double().abs()
        close(y, yr, dtype, ymag, c, ("y", act, pad, off))
        if z:
            close(got[1], zr, dtype, mag, c, ("z", act, pad, off))
    assert A.device_error() == A.OK


def linear_grad_check(A, dy, x, w, z, act, dtype, dw_type, got):
    dx, dw, db = got
    slope = act_slope_ref(z.double(), act) if act else 1.0
    dz = dy.double() * slope
    rows, n, k = dy.shape[0], w.shape[0], w.shape[1]
    # dz is rounded to the operands' type (U |dz|); its own arithmetic: 16 roundings
    u = U[dtype] if act else 0.0
    sl = 16 * E * (dy.double().abs() * (2 * z.double().abs() + 2)) if act else torch.zeros_like(dz)
    dz_err = u * dz.abs() + sl + (2.0 ** -25 if act and dtype == "f16" else 0.0)
    if dx is not None:
        close(dx, dz @ w.double(), dtype, dz.abs() @ w.double().abs() + dz_err @ w.double().abs() / E,
              2 * (n / 16 + 4), "dx")
    if dw is not None:
        # an fp32 result is taken in chains of 512, rounded to nearest: 2 E times 32 steps
        # and one E per chain
        c = 2 * 36 + rows / 512 + 8 if dw_type == "f32" else 2 * (rows / 16 + 4)
        close(dw, dz.t() @ x.double(), dw_type, dz.abs().t() @ x.double().abs() + dz_err.t() @ x.double().abs() / E / c,
              c, "dweight")
    if db is not None:
        close(db, dz.sum(0), "f32", dz.abs().sum(0) + sl.sum(0) / E / 128, 128, "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", LINEAR_SHAPES + [(5000, 256, 200), (9000, 64, 72)], ids=lambda s: "x".join(map(str, s)))
def test_linear_backward(A, shape, transposed, dtype):
    rows, n, k = shape
    for i, (act, dw_type, pad, off) in enumerate([(None, "f32", 0, 0), ("relu2", dtype, 0, 0), ("gelu", "f32", 1, 1),
                                                  ("silu", dtype, 8, 0)]):
        dy = randn(1200 + i, rows, n, dtype=dtype, pad=pad, offset=off)
        x = randn(1300 + i, rows, k, dtype=dtype, pad=pad, offset=off)
        w = make_weight(1400 + i, n, k, dtype, transposed, pad, off)
        z = randn(1500 + i, rows, n, dtype=dtype, pad=pad) if act else None
        got = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=DT[dw_type])
        assert got[1].stride() == ((1, n) if transposed and n > 1 and k > 1 else got[1].stride())
        linear_grad_check(A, dy, x, w, z, act, dtype, dw_type, got)
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", [(8192, 2816, 768), (4096, 1024, 3000), (4099, 1027, 3001), (2500, 2304, 4200)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_backward_both_products(A, shape, transposed, dtype):
    """Sizes whose products share the device: a last turn of the first that is not full, the second in parts."""
    rows, n, k = shape
    for i, (act, dw_type) in enumerate([("relu2", "f32"), (None, dtype)]):
        dy, x = randn(1210 + i, rows, n, dtype=dtype), randn(1310 + i, rows, k, dtype=dtype)
        w = make_weight(1410 + i, n, k, dtype, transposed)
        z = randn(1510 + i, rows, n, dtype=dtype) if act else None
        got = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=DT[dw_type])
        linear_grad_check(A, dy, x, w, z, act, dtype, dw_type, got)
        # which pairs start first does not show
        for _ in range(3):
            again = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=DT[dw_type])
            assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 2, 3])
@pytest.mark.parametrize("shape", [(1, 7), (5, 8), (3, 24570), (3, 24060), (100, 12301), (70, 12030), (2816, 768), (768, 2816), (5001, 520), (12007, 1030),
                                   (9800, 264), (4096, 4096), (4100, 4100)], ids=lambda s: "x".join(map(str, s)))
def test_linear_tokens(A, shape, rows, dtype):
    n, k = shape
    x, w = randn(1230, rows, k, dtype=dtype), randn(1231, n, k, scale=k ** -0.5, dtype=dtype, pad=(-k) % 8)
    b, r = randn(1232, n, scale=0.3), randn(1233, rows, n, dtype=dtype)
    y, z = A.linear_forward(x, w, b, activation="silu", residual=r, save_preact=True)
    zr = x.double() @ w.double().t() + b.double()
    mag = x.double().abs() @ w.double().abs().t() + b.double().abs()
    c = 2 * (k / 16 + 4)
    close(z, zr, dtype, mag, c, "z")
    close(y, act_ref(zr, "silu") + r.double(), dtype, 1.2 * mag + 8 * (zr.abs() + zr.square()) + r.double().abs(), c, "y")
    plain = A.linear_forward(x, w)
    close(plain, zr - b.double(), dtype, mag, c, "plain")
    # a transposed bank's input gradient takes the same path
    dy = randn(1234, rows, n, dtype=dtype)
    wt = randn(1235, k, n, scale=k ** -0.5, dtype=dtype, pad=(-n) % 8).t()
    dx = A.linear_backward(dy, x, wt, need_dweight=False, bias_grad=False)[0]
    close(dx, dy.double() @ wt.double(), dtype, dy.double().abs() @ wt.double().abs(), 2 * (n / 16 + 4), "dx")
    assert A.device_error() == A.OK


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 17, 32, 70])
def test_linear_few_rows_of_wide_layers(A, rows, transposed):
    """More blocks of weight rows than SMs."""
    n, k = 20011, 200
    x = randn(1220, rows, k, dtype="bf16")
    w = make_weight(1221, n, k, "bf16", transposed, pad=5)
    b = randn(1222, n)
    y = A.linear_forward(x, w, b, activation="relu")
    ref = (x.double() @ w.double().t() + b.double()).clamp_min(0)
    mag = x.double().abs() @ w.double().abs().t() + b.double().abs()
    close(y, ref, "bf16", mag, 2 * (k / 16 + 4), "y")
    assert A.device_error() == A.OK


@pytest.mark.parametrize("act", ["relu", "relu2", "gelu", "gelu_tanh", "silu"])
def test_linear_activations(A, act):
    """Every activation forward and backward, around 0 and far out."""
    n = k = 64
    x = torch.linspace(-12, 12, 200 * 64, device="cuda").reshape(200, 64).bfloat16()
    w = torch.eye(64, device="cuda").bfloat16()
    y, z = A.linear_forward(x, w, activation=act, save_preact=True)
    assert torch.equal(z, x)
    ref = act_ref(x.double(), act)
    close(y, ref, "bf16", ref.abs() + x.double().abs(), 16, act)
    dy = torch.ones_like(x)
    got = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=torch.float32)
    linear_grad_check(A, dy, x, w, z, act, "bf16", "f32", got)


@pytest.mark.parametrize("shape", [(40, 96, 136), (3000, 300, 200), (20000, 96, 64)])
@pytest.mark.parametrize("dw_type", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_linear_accumulate(A, shape, dw_type, pad):
    """dweight and dbias added to what is there, once per call."""
    rows, n, k = shape
    dy, x = randn(1, rows, n, dtype="bf16", scale=0.1), randn(2, rows, k, dtype="bf16")
    w = randn(3, n, k, dtype="bf16")
    dw0, db0 = randn(4, n, k, dtype=dw_type, pad=pad), randn(5, n)
    dw, db = randn(4, n, k, dtype=dw_type, pad=pad), db0.clone()
    assert torch.equal(dw, dw0)
    A.linear_backward(dy, x, w, dweight=dw, dbias=db, accumulate=True, need_dx=False)
    p, q = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    c = 2 * 36 + rows / 512 + 8 if dw_type == "f32" else 2 * (rows / 16 + 4)
    close(dw, dw0.double() + p, dw_type, q + dw0.double().abs(), c, "dweight")
    close(db, db0.double() + dy.double().sum(0), "f32", db0.double().abs() + dy.double().abs().sum(0), 128, "dbias")


@pytest.mark.parametrize("rows", [1, 100, 700])
def test_linear_residual_in_place_and_subsets(A, rows):
    x, w, r = randn(1, rows, 136, dtype="bf16"), randn(2, 200, 136, dtype="bf16", scale=0.1), randn(3, rows, 200, dtype="bf16")
    want = A.linear_forward(x, w, residual=r)
    r2 = r.clone()
    assert torch.equal(A.linear_forward(x, w, residual=r2, out=r2), want)
    dy = randn(4, rows, 200, dtype="bf16")
    dx, dw, db = A.linear_backward(dy, x, w)
    assert torch.equal(A.linear_backward(dy, x, w, need_dweight=False, bias_grad=False)[0], dx)
    assert torch.equal(A.linear_backward(dy, x, w, need_dx=False, bias_grad=False)[1], dw)
    assert torch.equal(A.linear_backward(dy, x, w, need_dx=False, need_dweight=False)[2], db)
    wide = torch.zeros(rows, 3, 200, dtype=torch.bfloat16, device="cuda")  # a column block of a wider result
    A.linear_forward(x, w, residual=r, out=wide[:, 1])
    assert torch.equal(wide[:, 1], want) and not wide[:, 0].any() and not wide[:, 2].any()


@pytest.mark.parametrize("rows", [3, 300])
def test_linear_infinities_stay_in_their_rows(A, rows):
    x, w = randn(1, rows, 100, dtype="bf16"), randn(2, 90, 100, dtype="bf16")
    clean = A.linear_forward(x, w)
    x2 = x.clone()
    x2[1, 7], x2[2, 3] = math.inf, math.nan
    y = A.linear_forward(x2, w)
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()


def test_linear_gradient_against_differences(A):
    """The directional derivative of the plain forward in 64 bits against the gradients of
    the kernels, whose dz is rounded to bf16: 2^-8 of the terms' root sum of squares."""
    rows, n, k = 50, 40, 72
    x, w, b = randn(1, rows, k, dtype="bf16"), randn(2, n, k, dtype="bf16", scale=k ** -0.5), randn(3, n)
    dy = randn(4, rows, n, dtype="bf16")
    h = 1e-6
    for act in ("gelu", "silu", "gelu_tanh"):
        # z is stored in bf16, so the loss is taken around the stored z
        _, z = A.linear_forward(x, w, b, activation=act, save_preact=True)
        dx, dw, db = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=torch.float32)
        z0 = z.double()

        def loss(ex, ew, eb):
            dzv = (x.double() + ex) @ (w.double() + ew).t() + eb - x.double() @ w.double().t()
            return (act_ref(z0 + dzv, act) * dy.double()).sum()
        for g, i, shape in ((dx, 0, (rows, k)), (dw, 1, (n, k)), (db, 2, (n,))):
            v = randn(30 + i, *shape).double()
            up, dn = [0.0] * 3, [0.0] * 3
            up[i], dn[i] = h * v, -h * v
            num = float((loss(*up) - loss(*dn)) / (2 * h))
            terms = g.double() * v
            assert abs(float(terms.sum()) - num) < 2.0 ** -6 * float(terms.square().sum().sqrt()) + 1e-6, (act, i)


def test_linear_empty(A):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = randn(1, 32, 64, dtype="bf16")
    y = A.linear_forward(x, w)
    assert y.shape == (0, 32)
    dx, dw, db = A.linear_backward(y, x, w, dweight_dtype=torch.float32)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


# ---------------------------------------------------------------- token log probabilities
def logits(seed, rows, vocab, dtype, masked, pad=0, offset=0):
    x = randn(seed, rows, vocab, scale=2.5, dtype=dtype, pad=pad, offset=offset).clone() if not (pad or offset) else \
        randn(seed, rows, vocab, scale=2.5, dtype=dtype, pad=pad, offset=offset)
    if masked:
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        x.masked_fill_(torch.rand((rows, vocab), generator=g, device="cuda") < 0.4, -math.inf)
        x[rows // 2] = -math.inf
        if rows > 2:
            x[rows - 1] = torch.finfo(DT[dtype]).min  # a mask of the lowest value: uniform
    return x


def logprob_ref(x, t, top):
    x = x.double()
    lse = torch.logsumexp(x, 1)
    dead = torch.isneginf(lse)
    p = torch.softmax(x, 1).nan_to_num(0.0)
    lp = torch.log_softmax(x, 1)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    tok = torch.where(dead, lse, lp.gather(1, t.clamp_min(0).long()[:, None])[:, 0])
    tok = torch.where(t < 0, torch.zeros_like(tok), tok)
    order = torch.sort(x, dim=1, descending=True, stable=True)  # equal values keep their columns' order
    val = torch.where(dead[:, None], torch.full_like(x, -math.inf), lp.gather(1, order.indices))
    return lse, ent, tok, val[:, :top], order.indices[:, :top]


LOGPROB_SHAPES = [(1, 1), (1, 2), (3, 7), (1, 50304), (2, 33), (5, 1000), (40, 5003), (160, 4096), (1, 131072), (9, 50257),
                  (700, 640)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("shape", LOGPROB_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_logprob_forward(A, shape, masked, dtype):
    rows, vocab = shape
    for k, (pad, off, top, tt) in enumerate([(0, 0, 0, torch.int64), (3, 1, min(32, vocab), torch.int32),
                                             (8, 0, min(5, vocab), torch.int64)]):
        x = logits(50 + k, rows, vocab, dtype, masked, pad, off)
        g = torch.Generator(device="cuda").manual_seed(60 + k)
        t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(tt)
        t[rows // 3] = -1
        lp, ent, lse, tv, ti = A.token_logprobs(x, t, top=top)
        rl, re, rt, rv, ri = logprob_ref(x, t, top)
        for got, ref, what in ((lse, rl, "lse"), (ent, re, "entropy"), (lp, rt, "logprob")) + \
                (((tv, rv, "top"),) if top else ()):
            inf = torch.isinf(ref)
            assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].double(), ref[inf]), what
            # a sum of 2^y: the exponent's rounding (|x - m| up to 60, times log2 e) and chains
            # of at most 131072 / (8 * 256) = 64 additions per thread, 8 more joins; the entropy
            # adds the same terms times |x - m| <= log(vocab) + entropy, at most 30
            fin = ~inf
            scale = 1.0 + ref.abs() + (x.double().masked_fill(torch.isinf(x), 0).abs().amax(1)
                                       if what != "top" else 0 * ref)
            if what == "entropy":
                scale = 30.0 + 0 * ref
            if what == "logprob" or what == "top":
                scale = 30.0 + ref.abs()
            close(got[fin], ref[fin], "f32", scale[fin], 192, what)
        if top:
            assert torch.equal(ti.long(), ri)
    assert A.device_error() == A.OK


def test_logprob_ties_and_signed_zero(A):
    """Equal values, +0 and -0 among them, come in the order of their columns."""
    x = torch.full((4, 3000), -3.0, device="cuda", dtype=torch.bfloat16)
    x[0, 77::100] = 2.0
    x[1, 5], x[1, 2999], x[1, 1500] = -0.0, 0.0, 0.0
    x[2] = 1.0
    x[3, 2000:] = -math.inf
    x[3, :2000] = -math.inf
    x[3, 2990] = 0.5
    _, _, _, tv, ti = A.token_logprobs(x, top=20)
    assert ti[0].tolist() == list(range(77, 77 + 2000, 100))
    assert ti[1].tolist()[:5] == [5, 1500, 2999, 0, 1]
    assert ti[2].tolist() == list(range(20))
    assert ti[3].tolist() == [2990] + list(range(19)) and torch.isinf(tv[3, 1:]).all() and float(tv[3, 0]) == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 400])
def test_logprob_top_of_uneven_rows(A, rows, dtype):
    """More candidates than a list holds: few distinct values, a few valid tokens, the large values all in one
    lane's vectors."""
    vocab = 40007
    x = torch.full((rows, vocab), -2.0, device="cuda", dtype=DT[dtype])
    col = torch.arange(vocab, device="cuda")
    unit = 16 // x.element_size()
    kinds = [torch.where(col % 3 == 1, 1.0, -1.0),                                             # two values
             torch.where((col > 30000) & (col < 30007), 0.25 * (col % 4), -math.inf),          # six tokens, with ties
             torch.where(col // unit % 32 == 5, (col * 7919 % 20011 - 10005) / 1024.0, -20.0),  # one lane in 32
             torch.where(col == vocab - 1, 3.0, torch.where(col == 0, 2.0, 0.0)),              # the ends of the row
             torch.where(col // unit % 32 == 9, 5.0, -20.0 + (col % 64) / 64.0)]               # equal values in one lane
    for r in range(rows):
        x[r] = kinds[r % 5]
    for k, off in enumerate((0, 1, 3)):  # three alignments
        y = x[:, off:]
        for top in (1, 8, 32):
            _, _, _, tv, ti = A.token_logprobs(y, top=top)
            val, idx = torch.sort(y.double(), dim=1, descending=True, stable=True)
            assert torch.equal(ti.long(), idx[:, :top]), (off, top)
    for kind in kinds:  # and alone
        y = kind.to(DT[dtype])[None]
        _, idx = torch.sort(y.double(), dim=1, descending=True, stable=True)
        assert torch.equal(A.token_logprobs(y, top=20)[4].long(), idx[:, :20])


def test_logprob_bad_rows_and_targets(A):
    x = randn(1, 6, 1000)
    x[1, 10], x[2, 20] = math.nan, math.inf
    t = torch.tensor([3, 10, 20, 1000, -100, 5], device="cuda")
    lp, ent, lse, tv, ti = A.token_logprobs(x, t, top=3)
    assert torch.isnan(lp[[1, 2, 3]]).all() and torch.isnan(lse[[1, 2]]).all() and torch.isnan(tv[[1, 2]]).all()
    assert not torch.isnan(lp[[0, 4, 5]]).any() and float(lp[4]) == 0.0 and not torch.isnan(lse[[0, 3, 4, 5]]).any()
    gl = torch.ones(6, device="cuda")
    d = A.token_logprobs_backward(x, t, lse, gl)
    assert torch.isnan(d[[1, 2, 3]]).all() and not d[4].any() and not torch.isnan(d[[0, 5]]).any()


def logprob_grad_ref(x, t, lse, ent, gl, gh):
    x, lse = x.double(), lse.double()[:, None]
    dead = torch.isneginf(lse)
    logp = x - torch.where(dead, torch.zeros_like(lse), lse)
    p = torch.exp(logp).masked_fill(dead, 0.0)
    u = torch.where(t >= 0, gl.double(), torch.zeros_like(gl.double()))[:, None] if gl is not None else 0.0
    d = -p * u
    mag = p * (abs(u) if gl is not None else 0.0)
    if gh is not None:
        s = torch.where(p > 0, logp + ent.double()[:, None], torch.zeros_like(p))
        d = d - gh.double()[:, None] * p * s
        mag = mag + gh.double().abs()[:, None] * p * (torch.where(p > 0, logp.abs(), 0 * p) + ent.double()[:, None])
    if gl is not None:
        hit = (torch.arange(x.shape[1], device=x.device)[None] == t.long()[:, None]) & ~dead
        d, mag = d + hit * u, mag + hit * abs(u)
    return d, mag


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("shape", LOGPROB_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_logprob_backward(A, shape, masked, dtype):
    rows, vocab = shape
    for k, (pad, off, out_off, with_gl, with_gh) in enumerate([(0, 0, 0, True, False), (3, 1, 0, True, True),
                                                               (8, 0, 8, False, True), (7, 1, 1, True, True)]):
        x = logits(70 + k, rows, vocab, dtype, masked, pad, off)
        g = torch.Generator(device="cuda").manual_seed(80 + k)
        t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        t[rows // 3] = -1
        _, ent, lse, _, _ = A.token_logprobs(x, t)
        gl = randn(90 + k, rows) if with_gl else None
        gh = randn(95 + k, rows) if with_gh else None
        out = torch.empty((rows, vocab + 9), dtype=DT[dtype], device="cuda")[:, out_off:out_off + vocab] if k else None
        d = A.token_logprobs_backward(x, t, lse, gl, entropy=ent, grad_entropy=gh, out=out)
        ref, mag = logprob_grad_ref(x, t, lse, ent, gl, gh)
        # p = 2^y: y's rounding is |x - lse| <= 60 of E, twice, over log2 e
        close(d, ref, dtype, mag, 256, (pad, off))
        if k == 0:
            y = x.clone()
            assert torch.equal(A.token_logprobs_backward(y, t, lse, gl, out=y), d)
    assert A.device_error() == A.OK


def test_logprob_gradient_against_differences(A):
    x = randn(1, 4, 301)
    t = torch.tensor([5, 300, 0, 77], device="cuda")
    lp, ent, lse, _, _ = A.token_logprobs(x, t)
    gl, gh = randn(2, 4), randn(3, 4)
    d = A.token_logprobs_backward(x, t, lse, gl, entropy=ent, grad_entropy=gh)
    v, h = randn(4, 4, 301).double(), 1e-5

    def loss(y):
        _, e, k, _, _ = logprob_ref(y, t, 0)
        return (k * gl.double()).sum() + (e * gh.double()).sum()
    num = (loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)
    assert abs(float((d.double() * v).sum() - num)) < 1e-4 * float((d.double() * v).abs().sum())


def test_logprob_empty(A):
    x = torch.empty((0, 100), device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    lp, ent, lse, tv, ti = A.token_logprobs(x, t, top=4)
    assert lp.shape == (0,) and ti.shape == (0, 4)
    assert A.token_logprobs_backward(x, t, lse, lp).shape == (0, 100)


# ---------------------------------------------------------------- streams, graphs, long arrays
def run_all(A, s):
    x, w, b, t = s
    h, mean, rstd = A.layernorm_forward(x, b[:136].float().contiguous())
    y, z = A.linear_forward(h, w, b, activation="relu2", save_preact=True)
    lp, ent, lse, _, _ = A.token_logprobs(y, t)
    dl = A.token_logprobs_backward(y, t, lse, torch.full_like(lp, -0.01))
    dx, dw, db = A.linear_backward(dl, h, w, preact=z, activation="relu2", dweight_dtype=torch.float32)
    return (h, y, lp, ent, dl, dw, db) + A.layernorm_backward(dx, x, mean, rstd)


def block_inputs(rows=700):
    return (randn(1, rows, 136, dtype="bf16"), randn(2, 2000, 136, dtype="bf16", scale=0.1),
            randn(3, 2000, dtype="bf16"), torch.arange(rows, device="cuda") % 2000)


@pytest.mark.parametrize("rows", [4, 700, 5000])
def test_same_bits_every_time_and_on_other_streams(A, rows):
    s = block_inputs(rows)
    want = run_all(A, s)
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run_all(A, s), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_all(A, s)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = A.linear_forward(s[0], s[1], s[2], stream=side)   # the stream as an argument
    side.synchronize()
    assert torch.equal(y, A.linear_forward(s[0], s[1], s[2]))


def test_graph_capture(A):
    s = block_inputs()
    want = run_all(A, s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run_all(A, s)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert A.device_error() == A.OK


def test_offsets_past_32_bits(A):
    """Rows whose element offsets pass 2^31: a strided view of one large buffer."""
    ld, rows, n = 1 << 28, 10, 768
    buf = torch.empty(ld * (rows - 1) + n, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (rows, n), (ld, 1))
    x.copy_(randn(1, rows, n, dtype="bf16"))
    c = x.contiguous()
    w = randn(2, 300, n, dtype="bf16", scale=0.05)
    t = torch.arange(rows, device="cuda")
    assert torch.equal(A.layernorm_forward(x)[0], A.layernorm_forward(c)[0])
    assert torch.equal(A.linear_forward(x, w), A.linear_forward(c, w))
    a, b = A.token_logprobs(x, t, top=3), A.token_logprobs(c, t, top=3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    lse = a[2]
    assert torch.equal(A.token_logprobs_backward(x, t, lse, lse), A.token_logprobs_backward(c, t, lse, lse))
