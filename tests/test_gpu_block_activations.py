"""GPU tests of the linear layer's activations and their slopes over the whole range of z, with bars
relative to the value itself, so that a tail counts as much as the middle."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, DT, E, U  # noqa: E402,F401  (A: fixture)

TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the spacing of the type's subnormals


def every_value(dtype, most):
    """Every finite value of the type with |z| <= most, in rows of 64 (the last one filled up with zeros)."""
    z = torch.arange(-(1 << 15), 1 << 15, device="cuda").to(torch.int16).view(DT[dtype])
    z = z[z.abs() <= most]
    return torch.nn.functional.pad(z, (0, -z.numel() % 64)).reshape(-1, 64)


def reference(z, act):
    """(value, slope, the size of the slope's terms) in 64 bits."""
    z = z.double()
    phi, cdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z * cdf, cdf + z * phi, cdf + z.abs() * phi


def outputs(A, x, act):  # noqa: F811
    """act(x) through a product with the identity, by each of the layer's kernels."""
    w = torch.eye(64, device="cuda").to(x.dtype)
    some = x[::max(1, x.shape[0] // 9)]
    yield x, A.linear_forward(x, w, activation=act)                                          # tiles
    yield some, torch.cat([A.linear_forward(r[None], w, activation=act) for r in some])      # one token
    for i in range(0, x.shape[0], 17 * 16):
        yield x[i:i + 17], A.linear_forward(x[i:i + 17], w, activation=act)                  # few rows


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act,most", [("gelu", 13.0)])
def test_activation_tails(A, act, most, dtype):  # noqa: F811
    """Every value within its own rounding and a relative error of the fp32 arithmetic: 48 E for the
    reciprocal, the polynomial and the products, 2 z^2 E for the exponential of z^2 / 2."""
    x = every_value(dtype, most)
    for z, y in outputs(A, x, act):
        ref = reference(z, act)[0]
        bar = (U[dtype] + E * (48 + 2 * z.double().square())) * ref.abs() + TINY[dtype]
        err = (y.double() - ref).abs()
        assert (err <= bar).all(), (float((err / bar.clamp_min(1e-300)).max()), z[err > bar][:5].tolist())
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act,most", [("gelu", 13.0)])
def test_slope_tails(A, act, most, dtype):  # noqa: F811
    """The bias's gradient of one row with dy = 1 is the slope itself in fp32."""
    z = every_value(dtype, most).reshape(1, -1)
    n = z.shape[1]
    x, w = torch.zeros((1, 8), device="cuda", dtype=z.dtype), torch.zeros((n, 8), device="cuda", dtype=z.dtype)
    _, _, db = A.linear_backward(torch.ones_like(z), x, w, preact=z, activation=act, need_dx=False, need_dweight=False)
    _, ref, size = reference(z[0], act)
    bar = E * (48 + 2 * z[0].double().square()) * size + 2.0 ** -148
    err = (db.double() - ref).abs()
    assert (err <= bar).all(), (float((err / bar).max()), z[0][err > bar][:5].tolist())
    assert A.device_error() == A.OK


def sigmoid_parts(z, act):
    """(u, du/dz, e^-|u| / (1 + e^-|u|) on either side) of z sigmoid(u(z)) in 64 bits."""
    z = z.double()
    u, du = z, torch.ones_like(z)
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        u, du = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z)
    return u, du, 1 / (1 + torch.exp(-u)), 1 / (1 + torch.exp(u))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_tanh_slope_far_out(A, dtype):  # noqa: F811
    """Every finite value of the type from |z| = 12 on, where the slope is 0 or 1 to the last bit."""
    z = every_value(dtype, math.inf).reshape(1, -1)
    z = z[(z.abs() >= 12) & torch.isfinite(z)][None]
    n = z.shape[1]
    x, w = torch.zeros((1, 8), device="cuda", dtype=z.dtype), torch.zeros((n, 8), device="cuda", dtype=z.dtype)
    _, _, db = A.linear_backward(torch.ones_like(z), x, w, preact=z, activation="gelu_tanh", need_dx=False, need_dweight=False)
    assert torch.equal(db, (z[0] > 0).float()), db[db != (z[0] > 0)][:5]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_sigmoid_tails(A, act, dtype):  # noqa: F811
    """Value and slope of every finite value of the type.

    u(z) takes at most 6 roundings (E |u| each, as an exponent), the exponential 2 (2 + 1.173 |u|) E,
    the reciprocal, the products and the sum 12 E; beyond |u| = 110 it is 0.  Below 2^-126 the
    exponential is off by up to 2^-149, times what it is multiplied with."""
    every = every_value(dtype, math.inf)
    every = torch.where(torch.isfinite(every), every, torch.zeros_like(every))

    def terms(z):
        u, du, s, c = sigmoid_parts(z, act)
        z, far = z.double(), u.abs().clamp_max(110.0)
        # (far out, where s c is 0, its factor z du is not taken into account)
        return z, du, s, c, E * (16 + 9 * far), torch.where(u.abs() < 110, 1 + z.abs() * du, torch.ones_like(z))
    for x, y in outputs(A, every, act):
        z, du, s, c, rel, lost = terms(x)
        ref = z * s
        bar = (U[dtype] + rel) * ref.abs() + TINY[dtype] + 2.0 ** -148 * (1 + z.abs().clamp_max(110.0))
        err = (y.double() - ref).abs()
        assert (err <= bar).all(), (float((err / bar).max()), x[err > bar][:5].tolist())
    x = every.reshape(1, -1)
    n = x.shape[1]
    _, _, db = A.linear_backward(torch.ones_like(x), torch.zeros((1, 8), device="cuda", dtype=x.dtype),
                                 torch.zeros((n, 8), device="cuda", dtype=x.dtype), preact=x, activation=act,
                                 need_dx=False, need_dweight=False)
    z, du, s, c, rel, lost = terms(x[0])
    inner = torch.where(s * c == 0, torch.zeros_like(z), z * c * du)
    ref = s + s * inner
    bar = 2 * rel * (s + s * inner.abs()) + 2.0 ** -147 * lost
    err = (db.double() - ref).abs()
    assert (err <= bar).all(), (float((err / bar).max()), x[0][err > bar][:5].tolist())
    assert A.device_error() == A.OK


@pytest.mark.parametrize("act", ["relu", "relu2", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows", [1, 300])
def test_nan_in_z_stays_nan(A, rows, act):  # noqa: F811
    """A NaN in z gives NaN in y, and in every gradient it takes part in."""
    x = torch.ones((rows, 64), device="cuda", dtype=torch.bfloat16)
    x[rows // 2, 5] = math.nan
    w = torch.eye(64, device="cuda").bfloat16()
    y = A.linear_forward(x, w, activation=act)
    assert torch.isnan(y[rows // 2]).all() and int(torch.isnan(y).sum()) == 64  # (each sum takes 0 * NaN)
    z = torch.ones((rows, 64), device="cuda", dtype=torch.bfloat16)
    z[rows // 2, 5] = math.nan
    ones = torch.ones_like(z)
    dx, dw, db = A.linear_backward(ones, ones, w, preact=z, activation=act)
    assert torch.isnan(dx[rows // 2]).all() and int(torch.isnan(dx).sum()) == 64
    assert torch.isnan(dw[5]).all() and int(torch.isnan(dw).sum()) == 64
    assert torch.isnan(db[5]) and int(torch.isnan(db).sum()) == 1


@pytest.mark.parametrize("rows", [3, 300])
def test_dz_beyond_fp16(A, rows):  # noqa: F811
    """A dz that fp16 does not hold is infinite in the products' operands, and stays in the gradients it
    takes part in; the bias's gradient is a sum of the unrounded values."""
    dy, z = torch.ones((rows, 64), device="cuda").half(), torch.ones((rows, 64), device="cuda").half()
    dy[1, 7], z[1, 7] = 300.0, 200.0                       # dz = 300 * 2 * 200 = 120000
    x, w = torch.ones((rows, 64), device="cuda").half(), torch.ones((64, 64), device="cuda").half()
    dx, dw, db = A.linear_backward(dy, x, w, preact=z, activation="relu2", dweight_dtype=torch.float32)
    assert torch.isinf(dx[1]).all() and int(torch.isinf(dx).sum()) == 64
    assert torch.isinf(dw[7]).all() and int(torch.isinf(dw).sum()) == 64
    assert float(db[7]) == 120000.0 + 2 * (rows - 1) and not torch.isnan(dx).any() and not torch.isnan(dw).any()
