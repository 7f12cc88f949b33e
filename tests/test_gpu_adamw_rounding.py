"""GPU tests of the rounding of AdamW's steps with 8-bit states, whose quotients and roots are not the
general operations in the middle of the range: bit for bit against numpy's fp32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_adamw import A, F, HP, ROOTS, Case, encode, run  # noqa: E402,F401


@pytest.mark.parametrize("small", [-103, -110, -126, -140, -149], ids=lambda e: f"2^{e}")
@pytest.mark.parametrize("eps", [1e-8, 1e-15, 1.0])
def test_first_moments_of_almost_nothing(A, small, eps):  # noqa: F811
    """First moments down to the smallest value, beside zeros and ordinary ones: from the codes, and
    from gradients alone.  The parameters are 0, so that a step shows its quotient's last bit."""
    n = 256 * 24
    c = Case(A, 31, n, "f32", "f32", 8)
    rng = np.random.default_rng(32)
    m = (np.ldexp(rng.uniform(1, 2, n), small) * rng.choice([-1.0, 0.0, 1.0], n)).astype(F)
    m[256 * 8:256 * 12:7] = 1e-3  # whole ranges in one block
    g = np.where(rng.random(n) < 0.5, 0.0, np.ldexp(rng.uniform(1, 2, n), small + 1)).astype(F)
    r = (10.0 ** rng.uniform(-6, 0, n)).astype(F)
    rc, rs = encode(r, True)
    ms = np.abs(m.reshape(-1, 256)).max(1) * F(1 / 448)  # (the operator's own states hold nothing below 2^-100)
    q = m.reshape(-1, 256).astype(np.float64) / np.where(ms > 0, ms, np.inf)[:, None]
    mc = torch.from_numpy(np.clip(q, -448, 448).reshape(-1).astype(F)).to(torch.float8_e4m3fn)
    c.m.copy_(mc)
    c.v.copy_(torch.from_numpy(rc))
    c.scales.copy_(torch.from_numpy(np.stack([ms, rs])))
    c.p.zero_()
    c.g.copy_(torch.from_numpy(g))
    hp = dict(HP, eps=eps, grad_scale=1.0, lr=1e20)
    want = c.expect(A, hp)
    assert (want[0] != 0).any()
    run(A, [c], hp)
    c.check(want, (small, eps))


@pytest.mark.parametrize("beta2", [0.95, 1 - 1e-7, 1 - 1e-12])
def test_quotients_below_the_normal_values(A, beta2):  # noqa: F811
    """Small moments over large denominators: in the first step the root's factor is up to a million."""
    n = 256 * 16
    c = Case(A, 41, n, "f32", "f32", 8)
    rng = np.random.default_rng(42)
    c.m.view(torch.uint8).zero_(), c.scales[0].zero_()
    rc, rs = encode((2.0 ** rng.uniform(6, 12.9, n)).astype(F), True)
    c.v.copy_(torch.from_numpy(rc))
    c.scales[1].copy_(torch.from_numpy(rs))
    c.p.zero_()
    c.g.copy_(torch.from_numpy((2.0 ** rng.uniform(-100, -80, n)).astype(F)))
    hp = dict(HP, step=1, beta2=beta2, grad_scale=1.0, lr=1e25, eps=1e-8)
    want = c.expect(A, hp)
    run(A, [c], hp)
    c.check(want, beta2)


class Quotients:
    """A step of 2^24 values that leaves -m / (sqrt(v) + eps) as the parameters: lr, root and decay are 1, p is 0.
    With beta1 = 0 m is the gradient, and with beta2 = 1/2 v = root^2 scale^2 / 2 + g^2 / 2."""
    N, EPS = 1 << 24, F(2.0 ** -60)

    def __init__(self):
        self.p, self.g = torch.zeros(self.N, device="cuda"), torch.empty(self.N, device="cuda")
        self.m = torch.zeros(self.N, device="cuda", dtype=torch.float8_e4m3fn)
        self.v = torch.empty(self.N, device="cuda", dtype=torch.uint8)
        self.scales = torch.zeros(2, self.N // 256, device="cuda")

    def v_of(self, codes, scale, g):
        r = (ROOTS[codes].reshape(-1, 256) * scale[:, None]).reshape(-1)
        return (r * r) * F(0.5) + (g * F(0.5)) * g

    def check(self, A, codes, scale, g):  # noqa: F811
        want = -(g / (np.sqrt(self.v_of(codes, scale, g)) + self.EPS))
        self.p.zero_(), self.m.view(torch.uint8).zero_()
        self.g.copy_(torch.from_numpy(g))
        self.v.copy_(torch.from_numpy(codes))
        self.scales[0].zero_()
        self.scales[1].copy_(torch.from_numpy(scale))
        A.adamw_step([self.p], [self.g], [self.m], [self.v], 1.0, 1, beta1=0.0, beta2=0.5, eps=float(self.EPS),
                     scales=[self.scales], scalars=torch.ones(4, device="cuda"))
        got = self.p.cpu().numpy()
        # (0 - u times 1: a u of 0 leaves +0)
        assert np.array_equal(got, want + F(0))


def test_roots_of_every_significand(A):  # noqa: F811
    """v: every fp32 value from 1 to 4, so every significand at either parity of the exponent, and with
    their roots every significand of the divisor.  The codes give the largest y^2 / 2 below v (y of six
    bits), the gradient the rest, to less than half of v's last place."""
    q = Quotients()
    v = np.concatenate([np.arange(1 << 23, dtype=np.uint32) + (e << 23) for e in (127, 128)]).view(F)
    codes = np.arange(256)
    squares = np.where(codes < 64, (ROOTS.astype(np.float64) / 16) ** 2 / 2, 1e9)
    at = (np.searchsorted(squares, v.astype(np.float64), side="right") - 1).astype(np.uint8)
    g = np.sqrt(2 * (v.astype(np.float64) - squares[at])).astype(F)
    scale = np.full(q.N // 256, 1 / 16, F)
    assert np.array_equal(q.v_of(at, scale, g), v)
    q.check(A, at, scale, g)


def middle_dividends(d):
    """For divisors d with an odd last bit the dividends (near 2^-20 d) whose quotients are as near to the
    middle between two fp32 values as any: with D the significand as an integer, t D = -1 or 1 (mod 2^25)
    for an odd t of 25 bits, so (t D + 1 or - 1) / 2^25 is a whole number, and over D it is t / 2^25 to 2^-48."""
    fraction, exponent = np.frexp(d.astype(np.float64))
    D = np.ldexp(fraction, 24).astype(np.uint64)
    inverse = D.copy()  # of odd D: Newton's iteration doubles the correct bits, three at first
    for _ in range(4):
        inverse *= np.uint64(2) - D * inverse
    t = inverse & np.uint64((1 << 25) - 1)
    up = t < 1 << 24  # t or its negative has 25 bits
    t = np.where(up, np.uint64(1 << 25) - t, t)
    whole = D * t + np.where(up, np.uint64(1), np.uint64(0)) - np.where(up, np.uint64(0), np.uint64(1))
    odd = D % 2 == 1
    assert not (whole[odd] % np.uint64(1 << 25)).any()
    return np.ldexp((whole >> np.uint64(25)).astype(np.float64), exponent - 24 - 20).astype(F), odd


@pytest.mark.parametrize("seed", [1, 2, 3, 4])
def test_quotients(A, seed):  # noqa: F811
    """2^24 divisors of dividends with random significands; with odd seeds the quotients of those divisors
    that allow it are next to the middle between two fp32 values."""
    q = Quotients()
    rng = np.random.default_rng(seed)
    codes = rng.integers(1, 256, q.N, dtype=np.uint8)
    scale = np.ldexp(rng.uniform(1, 2, q.N // 256), rng.integers(-40, -15, q.N // 256)).astype(F)
    zero = np.zeros(q.N, F)
    d = np.sqrt(q.v_of(codes, scale, zero)) + q.EPS
    g = d * np.ldexp(rng.uniform(1, 2, q.N), -20).astype(F)  # its square is lost beside v
    if seed % 2:
        hard, odd = middle_dividends(d)
        assert odd.mean() > 0.4
        g = np.where(odd, hard, g)
    assert np.array_equal(q.v_of(codes, scale, g), q.v_of(codes, scale, zero))
    q.check(A, codes, scale, g)
