"""GPU tests of the head's cross entropy at the ends of its range: long contractions, logits beyond what their
multiples of log2(e) resolve, row gradients that are not finite.  Against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, E, U, close, make_weight, randn  # noqa: E402,F401
from test_gpu_head import backward_check, make_targets  # noqa: E402


def uniform(seed, *shape, lo, hi, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo).to({"bf16": torch.bfloat16, "f16": torch.float16}[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 3, 16, 20, 32, 33, 300, 700])
@pytest.mark.parametrize("k", [512, 777, 4096, 16391, 65536])
def test_long_contractions(A, k, rows, transposed, dtype):  # noqa: F811
    """Products of one sign, where sums that are cut off drift the same way: the tensor cores' sums end after 1024
    terms and are added up rounded to nearest."""
    vocab = 1000
    x = uniform(1, rows, k, lo=0.5, hi=1.5, dtype=dtype)
    w = uniform(2, vocab, k, lo=5.0 / k, hi=15.0 / k, dtype=dtype)
    if transposed:
        w = w.t().contiguous().t()
    t = make_targets(3, rows, vocab)
    loss, lse = A.linear_cross_entropy(x, w, t)
    z = x.double() @ w.double().t()  # every product is positive: its own magnitude
    # chains of 64 steps at 2 E each and the chains' sum
    ez = (2 * (64 + 4) + k / 1024 + 8) * E * z
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    parts = math.ceil(vocab / 256) * 4
    bar = (p * ez).sum(1) + E * (4 + 2 + 24 + 11 * (parts / 8 + 9) + 4 * want.abs() + 4)  # forward_check's arithmetic
    assert ((lse.double() - want).abs() <= 1.01 * bar).all(), float(((lse.double() - want).abs() / bar).max())
    live = t >= 0
    at = t.clamp_min(0)[:, None]
    ref = want - z.gather(1, at)[:, 0]
    bar = bar + ez.gather(1, at)[:, 0] + 2 * E * ref.abs()
    assert ((loss.double() - ref).abs() <= 1.01 * bar)[live].all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("k", [1024, 1100, 16391, 65536])
def test_gradients_of_long_contractions(A, k, rows, transposed, dtype):  # noqa: F811
    """The gradient's logits are added up as the forward pass's, or the probabilities would not fit lse."""
    vocab = 1000
    x = uniform(1, rows, k, lo=0.5, hi=1.5, dtype=dtype)
    w = uniform(2, vocab, k, lo=5.0 / k, hi=15.0 / k, dtype=dtype)
    if transposed:
        w = w.t().contiguous().t()
    t, gl = make_targets(3, rows, vocab), randn(4, rows).abs() + 0.5
    _, lse = A.linear_cross_entropy(x, w, t)
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=torch.float32)
    z = x.double() @ w.double().t()
    ez = (2 * (64 + 4) + k / 1024 + 8) * E * z  # as above
    g = torch.where(t >= 0, gl.double(), 0.0)[:, None]
    p = torch.exp(z - lse.double()[:, None])
    d = (g * p).scatter_add(1, t.clamp_min(0)[:, None], -g)
    # backward_check's: p's and d's errors, the products' sums
    ep = p * (ez + 3 * E * (z + lse.double().abs()[:, None]) + 8 * E)
    ed = g * ep * 1.01 + (5 * E + U[dtype]) * d.abs()
    if dtype == "f16":
        ed = ed + 2.0 ** -38 * float(g.max()) * (g != 0)
    c = 2 * (vocab / 16 + 8)
    close(dx, d @ w.double(), dtype, d.abs() @ w.double() + ed @ w.double() / E / c, c, "dx")
    c = 2 * 36 + rows / 512 + 8
    close(dw, d.t() @ x.double(), "f32", d.abs().t() @ x.double() + ed.t() @ x.double() / E / c, c, "dweight")


SIZES = [3e3, 1.1e5, 1.3e6, 2.7e7, 7e8, 3.3e9, 5e12, 1e25, 3e37]


def one_above(rows, vocab, size, transposed, sign):
    """Logits of `size` or so, one per row above the others by a part in 128 at least; exact in fp32."""
    x = torch.zeros(rows, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(vocab, 64, device="cuda", dtype=torch.bfloat16)
    if transposed:
        w = torch.zeros(64, vocab, device="cuda", dtype=torch.bfloat16).t()
    x[:, 0] = 2.0 ** int(math.log2(size) / 2)
    w[:, 0] = sign * size / float(x[0, 0]) * (0.75 if sign > 0 else 1.5)
    w[vocab // 3, 0] = sign * size / float(x[0, 0])
    return x, w


@pytest.mark.parametrize("rows", [1, 2, 5, 40, 300, 900])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_large_logits(A, size, sign, transposed, rows):  # noqa: F811
    """The sum is of one exponential of 0 and nothing else, so lse is that logit, to the bit."""
    vocab = 700
    x, w = one_above(rows, vocab, size, transposed, sign)
    t = make_targets(3, rows, vocab)
    t[rows // 2] = vocab // 3
    loss, lse = A.linear_cross_entropy(x, w, t)
    z = x.float() @ w.float().t()
    most = z.amax(1)
    assert torch.equal(lse, most)
    want = torch.where(t >= 0, most - z.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0)
    assert torch.equal(loss, want)
    # d is -g and g, or 0 where the target is the largest
    gl = randn(4, rows).abs() + 0.5
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=torch.float32)
    d = torch.zeros(rows, vocab, device="cuda", dtype=torch.float64)
    live = torch.where(t >= 0, gl.double(), 0.0)
    d[:, vocab // 3] += live
    d.scatter_add_(1, t.clamp_min(0)[:, None], -live[:, None])
    # d: its rounding to bf16 and the factor's three; results: bf16's, or the sums'
    bar = 2.0 ** -8 + 16 * E
    ref, mag = d.t() @ x.double(), d.abs().t() @ x.double().abs()
    assert ((dw.double() - ref).abs() <= bar * mag + 80 * E * mag).all()
    ref, mag = d @ w.double(), d.abs() @ w.double().abs()
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (bar + 200 * E) * mag).all()


@pytest.mark.parametrize("rows", [1, 4, 40, 300])
def test_equal_large_logits(A, rows):  # noqa: F811
    """Half of the vocabulary at one large value: its logarithm is within lse's last places."""
    vocab = 700
    for size in SIZES:
        x, w = one_above(rows, vocab, size, False, 1)
        w[::2, 0] = w[vocab // 3, 0].clone()
        w[vocab // 3, 0] = 0.0  # (odd)
        z = float(x[0, 0]) * float(w[0, 0])
        _, lse = A.linear_cross_entropy(x, w)
        want = z + math.log(350.0)
        assert ((lse.double() - want).abs() <= E * want + 200 * E).all(), size


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_row_gradients_that_are_not_finite(A, bad):  # noqa: F811
    """fp16 holds the logits' gradients over the largest row gradient: of the finite ones, so that a row that is not
    does not take the others' digits."""
    rows, vocab, k = 90, 500, 64
    x, w = randn(1, rows, k, scale=2.0, dtype="f16"), make_weight(2, vocab, k, "f16", False)
    t, gl = make_targets(3, rows, vocab), randn(4, rows, scale=1e-4)
    _, lse = A.linear_cross_entropy(x, w, t)
    gl[11], t[11] = bad, 77
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl)
    keep = torch.arange(rows, device="cuda") != 11
    assert not torch.isfinite(dx[11]).any() and not torch.isfinite(dw[77]).any()
    backward_check(x[keep], w, t[keep], lse[keep], gl[keep], "f16", "f16", (dx[keep], None))
