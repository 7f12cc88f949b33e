"""GPU tests of AdamW over many tensors: bit for bit against numpy's fp32 (one rounding per operation,
in the documented order), and against 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
HP = dict(lr=3e-3, step=4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=0.5)
F = np.float32


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from polynomial_matrix_whitening_gb300 import anvil
    return anvil


def blocks(x):
    return np.concatenate([x, np.zeros(-len(x) % 256, x.dtype)]).reshape(-1, 256)


ROOTS = np.array([c if c < 16 else (16 + c % 16) * 2 ** (c // 16 - 1) for c in range(256)], F)


def encode(x, root):
    """(codes as stored, scale) of each block: nearest code from the table of values, ties to the even one."""
    top = F(ROOTS[-1] if root else 448)
    b = blocks(x)
    most = np.abs(b).max(1)
    most = np.where(most < F(2.0 ** -100), F(0), most)
    with np.errstate(all="ignore"):
        inverse = np.where(most > 0, top / most, F(0)).astype(F)
    scale = most * (F(1) / top)
    q = b * inverse[:, None]
    if not root:
        codes = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    else:
        middle = (ROOTS[1:].astype(np.float64) + ROOTS[:-1]) / 2
        c = np.searchsorted(middle, q.astype(np.float64))
        tie = (c < 255) & (middle[np.minimum(c, 254)] == q) & (c % 2 == 1)
        c = c + tie
        codes = np.where(q > 0, np.maximum(c, 1), 0).astype(np.uint8)
    return codes.reshape(-1)[:len(x)], scale


def decode(codes, scale, root):
    v = ROOTS[codes] if root else torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    return (blocks(v) * scale[:, None]).reshape(-1)[:len(codes)]


def values(t):
    """fp32 values of a tensor on the host."""
    return t.detach().float().cpu().numpy().reshape(-1)


def reference(A, p, g, m, v, hp, dtype=F):
    """p, m, v after a step and the root, elementwise in `dtype`."""
    k = {n: hp[n] for n in ("lr", "step", "beta1", "beta2", "weight_decay", "grad_scale")}
    if dtype is F:
        step_size, root, decay, scale = (F(x) for x in A.adamw_scalars(**k))
    else:
        step_size, root = hp["lr"] / (1 - hp["beta1"] ** hp["step"]), (1 - hp["beta2"] ** hp["step"]) ** -0.5
        decay, scale = 1 - hp["lr"] * hp["weight_decay"], hp["grad_scale"]
    b1, c1, b2, c2, eps = (dtype(x) for x in (hp["beta1"], 1 - hp["beta1"], hp["beta2"], 1 - hp["beta2"], hp["eps"]))
    p, g, m, v = (x.astype(dtype) for x in (p, g, m, v))
    g = g * scale
    m = m * b1 + g * c1
    v = v * b2 + (g * c2) * g
    r = np.sqrt(v)
    return p * decay - (m / (r * root + eps)) * step_size, m, v, r


class Case:
    """One tensor's arrays on the GPU, views into larger buffers with guard values on both sides."""

    def __init__(self, A, seed, count, param="f32", grad="f32", bits=32, offset=0):
        self.kind, self.count, self.bits = param, count, bits
        rng = np.random.default_rng(seed)
        self.buffers = []
        p = (rng.standard_normal(count) * 0.05).astype(F)
        g = torch.from_numpy((rng.standard_normal(count) * np.exp(rng.standard_normal(count) * 2) * 0.01).astype(F))
        m = (rng.standard_normal(count) * 0.004).astype(F)
        v = np.square(rng.standard_normal(count) * 0.01).astype(F)
        self.low = None
        if param == "split":
            bits32 = p.view(np.int32)
            self.low = self.put(torch.from_numpy((bits32 & 0xFFFF).astype(np.uint16).view(np.int16)), offset)
            self.p = self.put(torch.from_numpy((bits32 >> 16).astype(np.int16)).view(torch.bfloat16), offset)
        else:
            self.p = self.put(torch.from_numpy(p).to(DT[param]), offset)
        self.g = self.put(g.to(DT[grad]), offset)
        self.scales = None
        if bits == 32:
            self.m, self.v = self.put(torch.from_numpy(m), offset), self.put(torch.from_numpy(v), offset)
        else:
            mc, ms = encode(m, False)
            rc, rs = encode(np.sqrt(v), True)
            self.m = self.put(torch.from_numpy(mc).view(torch.float8_e4m3fn), offset)
            self.v = self.put(torch.from_numpy(rc), offset)
            self.scales = self.put(torch.from_numpy(np.concatenate([ms, rs])), offset).view(2, -1)
        self.before = [b.clone() for b, _, _ in self.buffers]

    def put(self, t, offset):
        full = torch.full((64 + offset + t.numel() + 64,), 7, dtype=torch.uint8, device="cuda").repeat(t.element_size())
        full = full.view(t.dtype)
        lo = 64 + offset
        full[lo:lo + t.numel()] = t.cuda()
        self.buffers.append((full.view(torch.uint8), lo * t.element_size(), (lo + t.numel()) * t.element_size()))
        return full[lo:lo + t.numel()]

    def master(self):
        if self.low is None:
            return values(self.p)
        hi = self.p.view(torch.int16).cpu().numpy().astype(np.int32) << 16
        return (hi | self.low.cpu().numpy().view(np.uint16).astype(np.int32)).view(F)

    def state(self):
        if self.bits == 32:
            m, v = values(self.m), values(self.v)
            return m, v
        s = self.scales.cpu().numpy()
        r = decode(self.v.cpu().numpy(), s[1], True)
        return decode(self.m.view(torch.uint8).cpu().numpy(), s[0], False), r * r

    def expect(self, A, hp=HP):
        """What the arrays will hold: (param or master, m or codes, v or codes, scales)."""
        m, v = self.state()
        with np.errstate(all="ignore"):
            p, m, v, r = reference(A, self.master(), values(self.g), m, v, hp)
        if self.kind in ("bf16", "f16"):
            p = values(torch.from_numpy(p).to(DT[self.kind]))
        if self.bits == 32:
            return p, m, v, None
        (mc, ms), (rc, rs) = encode(m, False), encode(r, True)
        return p, mc, rc, np.stack([ms, rs])

    def check(self, want, what=""):
        p, m, v, s = want
        assert np.array_equal(self.master(), p, equal_nan=True), (what, "param")
        if self.bits == 32:
            assert np.array_equal(values(self.m), m, equal_nan=True), (what, "exp_avg")
            assert np.array_equal(values(self.v), v, equal_nan=True), (what, "exp_avg_sq")
        else:
            assert np.array_equal(self.scales.cpu().numpy(), s, equal_nan=True), (what, "scales")
            assert np.array_equal(self.m.view(torch.uint8).cpu().numpy(), m), (what, "exp_avg")
            assert np.array_equal(self.v.cpu().numpy(), v), (what, "exp_avg_sq")
        for (now, lo, hi), before in zip(self.buffers, self.before):  # nothing beside the arrays
            assert torch.equal(now[:lo], before[:lo]) and torch.equal(now[hi:], before[hi:]), (what, "guard")


def run(A, cases, hp=HP, **kw):
    A.adamw_step([c.p for c in cases], [c.g for c in cases], [c.m for c in cases], [c.v for c in cases],
                 mantissas=[c.low for c in cases], scales=[c.scales for c in cases], **dict(hp, **kw))


KINDS = [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
         ("split", "bf16"), ("split", "f32")]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", KINDS, ids=lambda s: s)
def test_step_bit_for_bit(A, param, grad, bits):
    for offset in (0, 1, 3):
        cases = [Case(A, 10 * n + offset, n, param, grad, bits, offset) for n in (1, 3, 255, 256, 257, 1000, 4096, 4097, 70001)]
        want = [c.expect(A) for c in cases]
        run(A, cases)
        for c, w in zip(cases, want):
            c.check(w, (offset, c.count))
    assert A.device_error() == A.OK


@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")], ids=lambda s: s)
def test_step_against_64_bits(A, param, grad):
    c = Case(A, 5, 50001, param, grad, 32)
    p0, m0, v0 = c.master(), *c.state()
    p, m, v, r = reference(A, p0, values(c.g), m0, v0, HP, np.float64)
    run(A, [c])
    # fp32 roundings: the gradient's scale, a product each and the sum for m and v (and v's gradient
    # squared: the constants' roundings with them, at most 8 of 2^-24 of the terms); the root halves
    # v's, then two for the denominator, two for the quotient, two for the parameter
    E = 2.0 ** -24
    g = np.abs(values(c.g).astype(np.float64)) * HP["grad_scale"]
    mm, vm = np.abs(m0) * 0.9 + g * 0.1, v0 * 0.95 + g * g * 0.05
    assert (np.abs(values(c.m) - m) <= 8 * E * mm).all() and (np.abs(values(c.v) - v) <= 8 * E * vm).all()
    size = HP["lr"] / (1 - HP["beta1"] ** HP["step"]) / (np.sqrt(v) * (1 - HP["beta2"] ** HP["step"]) ** -0.5 + HP["eps"])
    bar = U[param] * np.abs(p) + 4 * E * np.abs(p0) + size * mm * 24 * E + (2.0 ** -25 if param == "f16" else 0)
    assert (np.abs(c.master() - p) <= bar * (1 + 1e-6)).all()


@pytest.mark.parametrize("eps", [1e-8, 0.0, 1e-20, 1e-30, 0.5, 100.0])
def test_extremes_bit_for_bit(A, eps):
    """Moments and gradients from 1e-30 to 1e30 and zeros, roots that belong to other moments, denominators of
    eps alone: quotients from 0 to infinity, as numpy has them.  (Where 8-bit states leave the middle
    of the range: |m| below 2^-102 is a last bit of nothing, so no value here is between 0 and 1e-30.)"""
    for bits in (8, 32):
        c = Case(A, 21, 256 * 40, "f32", "f32", bits)
        rng = np.random.default_rng(22)
        wide = lambda: (rng.choice([-1.0, 1.0], 256 * 40) * 10.0 ** np.repeat(rng.uniform(-30, 30, 40), 256)  # noqa: E731
                        * 10.0 ** rng.uniform(-1, 0, 256 * 40) * (rng.random(256 * 40) < 0.9)).astype(F)
        m, r, g = wide(), np.abs(wide()), wide()
        g[:256 * 20] = 0.0
        r = np.minimum(r, F(1e18))  # (squares stay finite)
        g = np.clip(g, F(-1e18), F(1e18))
        c.g.copy_(torch.from_numpy(g))
        if bits == 32:
            c.m.copy_(torch.from_numpy(m))
            c.v.copy_(torch.from_numpy(np.square(r)))
        else:
            (mc, ms), (rc, rs) = encode(m, False), encode(r, True)
            c.m.copy_(torch.from_numpy(mc).view(torch.float8_e4m3fn))
            c.v.copy_(torch.from_numpy(rc))
            c.scales.copy_(torch.from_numpy(np.stack([ms, rs])))
        hp = dict(HP, eps=eps)
        want = c.expect(A, hp)
        run(A, [c], hp)
        c.check(want, (bits, eps))


def test_steps_in_a_row(A):
    """Ten steps of 8-bit states from zero, each from what the last one left."""
    c = Case(A, 7, 5000, "f32", "f32", 8)
    c.m.view(torch.uint8).zero_(), c.v.zero_(), c.scales.zero_()
    for t in range(1, 11):
        hp = dict(HP, step=t)
        want = c.expect(A, hp)
        run(A, [c], hp)
        c.check(want, t)


def test_many_tensors_of_all_kinds(A):
    """More tensors than a launch takes, kinds and sizes mixed, some empty."""
    cases = [Case(A, 1000 + i, (i * 37) % 900, *KINDS[i % 9], bits=8 if i % 2 else 32, offset=i % 5) for i in range(1900)]
    want = [c.expect(A) if c.count else None for c in cases]
    run(A, cases)
    for i, (c, w) in enumerate(zip(cases, want)):
        if c.count:
            c.check(w, i)
    run(A, [Case(A, 1, 0)])


def test_values(A):
    cases = [Case(A, 50 + n, n, "f32", "f32", 8, offset) for n in (1, 256, 5000, 70001) for offset in (0, 1)]
    run(A, cases)
    ms, vs = A.adamw_values([c.m for c in cases], [c.v for c in cases], [c.scales for c in cases])
    for c, m, v in zip(cases, ms, vs):
        rm, rv = c.state()
        assert np.array_equal(values(m), rm) and np.array_equal(values(v), rv)


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite(A, bits):
    """A NaN or an infinity stays with its value (with its block's states in 8 bits); zeros, tiny and
    huge gradients."""
    c = Case(A, 9, 256 * 8, "f32", "f32", bits)
    c.g[3], c.g[256 + 9], c.g[512:768], c.g[768:1024] = math.nan, math.inf, 0.0, 1e-30
    c.g[1024:1280] *= 1e18  # squares stay finite
    if bits == 32:
        c.m[512:1024] = 0.0
        c.v[512:1024] = 0.0
    else:
        c.scales[:, 2:4] = 0.0
    want = c.expect(A)
    run(A, [c])
    if bits == 32:
        c.check(want)
        return
    p, m, v, s = want
    assert np.array_equal(c.master(), p, equal_nan=True)
    got_m, got_v = c.state()
    for b in range(8):
        at = slice(256 * b, 256 * b + 256)
        if b < 2:
            assert np.isnan(got_m[at]).all() and np.isnan(got_v[at]).all()
        else:
            assert np.array_equal(c.m.view(torch.uint8).cpu().numpy()[at], m[at])
            assert np.array_equal(c.v.cpu().numpy()[at], v[at])
    ms, vs = A.adamw_values([c.m], [c.v], [c.scales])
    assert torch.isnan(ms[0][:512]).all() and not torch.isnan(ms[0][512:]).any() and not torch.isnan(vs[0][512:]).any()


def test_a_root_above_zero_stays_above_zero(A):
    """States with roots a ten-millionth of their block's largest, below half the smallest code, and first
    moments that are not small beside each other.  As 0 such a root would make the next step m / eps =
    100 times lr; as the smallest code m / r is 0.5 at most, and falls from there: the gradient is 0."""
    m0, r0 = np.full(256, 1e-6, F), np.full(256, 1e-7, F)
    r0[0] = 1.0
    p, g = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    m, v, s = A.adamw_state(p, 8)
    (mc, ms), (rc, rs) = encode(m0, False), encode(r0, True)
    assert (rc[1:] == 1).all() and (mc != 0).all()
    m.copy_(torch.from_numpy(mc).view(torch.float8_e4m3fn)), v.copy_(torch.from_numpy(rc))
    s.copy_(torch.from_numpy(np.stack([ms, rs])))
    for t in range(100, 120):
        A.adamw_step([p], [g], [m], [v], 1e-3, t, scales=[s])
        assert (v[1:] == 1).all()
    assert 0 < float(p.abs().max()) < 20 * 0.55e-3


def test_graph_with_scalars(A):
    """A captured step follows the scalars on the device; two graphs share nothing."""
    cases = [Case(A, 60 + i, 3000, "split", "bf16", 8 if i else 32) for i in range(2)]
    scalars = torch.empty(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(A, cases, scalars=scalars)
    for t in (5, 6):
        hp = dict(HP, step=t, lr=1e-3 * t)
        scalars.copy_(torch.tensor(A.adamw_scalars(hp["lr"], t, 0.9, 0.95, 0.1, 0.5)))
        want = [c.expect(A, hp) for c in cases]
        graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            c.check(w, t)


def test_on_another_stream(A):
    c = Case(A, 70, 100001, "f32", "bf16", 8)
    want = c.expect(A)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(A, [c], stream=s)
    s.synchronize()
    c.check(want)


def test_parameters_that_require_grad(A):
    """A step in grad mode, and the graph that saved the old values refuses them."""
    w = torch.nn.Parameter(torch.ones(300, device="cuda"))
    y = (w * w).sum()
    m, v, _ = A.adamw_state(w)
    A.adamw_step([w], [torch.ones(300, device="cuda")], [m], [v], 1e-3, 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_refusals(A):
    c, d = Case(A, 1, 300, "bf16", "bf16", 8), Case(A, 2, 300)
    with pytest.raises(ValueError, match="grads must be"):
        A.adamw_step([c.p], [c.g.half()], [c.m], [c.v], 1e-3, 1, scales=[c.scales])
    with pytest.raises(ValueError, match="fp32, or 8-bit codes with scales"):
        A.adamw_step([c.p], [c.g], [c.m], [c.v], 1e-3, 1)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        A.adamw_step([c.p], [c.g], [d.m], [d.v], 1e-3, 1, scales=[c.scales])
    with pytest.raises(ValueError, match="size"):
        A.adamw_step([c.p], [c.g[:299]], [c.m], [c.v], 1e-3, 1, scales=[c.scales])
    with pytest.raises(ValueError, match="size"):
        A.adamw_step([c.p], [c.g], [c.m], [c.v], 1e-3, 1, scales=[c.scales[:, :1].contiguous()])
    with pytest.raises(ValueError, match="contiguous"):
        A.adamw_step([d.p[::2]], [d.g[:150]], [d.m[:150]], [d.v[:150]], 1e-3, 1)
    with pytest.raises(ValueError, match="mantissas"):
        A.adamw_step([d.p], [d.g], [d.m], [d.v], 1e-3, 1, mantissas=[torch.zeros(300, device="cuda", dtype=torch.int16)])
    with pytest.raises(A.AnvilError, match="ALIAS"):
        A.adamw_step([d.p, d.p], [d.g, d.g], [d.m, d.m], [d.v, d.v], 1e-3, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        A.adamw_step([d.p], [d.g.cpu()], [d.m], [d.v], 1e-3, 1)


def test_past_32_bit_offsets(A):
    """The last values of a tensor of more than 2^31."""
    n, tail = (1 << 31) + 300, 1000
    p, g = torch.zeros(n, device="cuda", dtype=torch.bfloat16), torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    m, v, s = A.adamw_state(p, 8)
    at = (n - tail) // 256 * 256
    keep = n - at
    ref = Case(A, 3, keep, "bf16", "bf16", 8)
    p[at:], g[at:] = ref.p, ref.g
    m.view(torch.uint8)[at:], v[at:], s[:, at // 256:] = ref.m.view(torch.uint8), ref.v, ref.scales
    want = ref.expect(A)
    A.adamw_step([p], [g], [m], [v], scales=[s], **HP)
    ref.p.copy_(p[at:])
    ref.m.view(torch.uint8).copy_(m.view(torch.uint8)[at:])
    ref.v.copy_(v[at:])
    ref.scales.copy_(s[:, at // 256:])
    ref.check(want)
    assert not p[:at].any()
