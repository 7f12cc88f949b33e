"""GPU tests of AdamW where a warp takes several blocks one after the other (each one's loads run beside the
arithmetic of the one before): bit for bit, as in test_gpu_adamw.py.  How many it takes follows from the blocks of a
call together, so a tensor of zeros beside the checked ones is enough."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_adamw import A, DT, KINDS, Case, run, values  # noqa: E402,F401

# chunks of 8, 16 and 32 blocks for a thread block's eight warps: up to one, two and four for a warp
FILL = {"one": 256, "two": 2600000, "four": 5100000}
COUNTS = (5, 256 * 8, 256 * 33 + 1, 256 * 64, 100003)


class Zeros:
    """A tensor of zeros, which a step leaves as it is."""

    def __init__(self, A, count, param, grad, bits, offset=0):
        new = lambda dtype: torch.zeros(count + offset, device="cuda", dtype=dtype)[offset:]  # noqa: E731
        self.p = new(torch.bfloat16 if param == "split" else DT[param])
        self.low = new(torch.int16) if param == "split" else None
        self.g = new(DT[grad])
        self.m, self.v = (new(torch.float8_e4m3fn), new(torch.uint8)) if bits == 8 else (new(torch.float32), new(torch.float32))
        self.scales = torch.zeros(2, -(-count // 256), device="cuda") if bits == 8 else None

    def check(self):
        for t in (self.p, self.low, self.m, self.v, self.scales):
            assert t is None or not t.view(torch.uint8).any()


def launches(A, call):
    call()  # (the first call loads the kernel)
    torch.cuda.synchronize()
    with A.profile() as prof:
        call()
        torch.cuda.synchronize()
    return [k for k, _ in prof.records]


@pytest.mark.parametrize("blocks", FILL)
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", KINDS, ids=lambda s: s)
def test_several_blocks_a_warp(A, param, grad, bits, offset, blocks):  # noqa: F811
    fill = Zeros(A, FILL[blocks] + 77, param, grad, bits, offset)
    cases = [Case(A, 100 + n + offset, n, param, grad, bits, offset) for n in COUNTS]
    want = [c.expect(A) for c in cases]
    run(A, cases[:2] + [fill] + cases[2:])
    for c, w in zip(cases, want):
        c.check(w, (c.count, blocks))
    fill.check()
    assert A.device_error() == A.OK


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("bf16", "bf16"), ("split", "bf16")], ids=lambda s: s)
def test_vectors_and_others_of_one_kind(A, param, grad, bits):  # noqa: F811
    """Many values on vector boundaries beside tensors off them take a launch each; a few join the others'."""
    for fill, want in ((330000, 2), (300000, 1)):  # 1216 blocks are 311296 values
        big = Zeros(A, fill, param, grad, bits)
        make = lambda: [Case(A, 7 + n + off, n, param, grad, bits, off) for off in (0, 1, 2) for n in (3, 257, 5000)]  # noqa: E731
        cases = make()
        expect = [c.expect(A) for c in cases]
        run(A, [big] + cases)
        for c, w in zip(cases, expect):
            c.check(w, (c.count, fill))
        big.check()
        again = make()
        assert launches(A, lambda: run(A, [big] + again)) == ["adamw"] * want


@pytest.mark.parametrize("blocks", FILL)
@pytest.mark.parametrize("offset", [0, 1])
def test_values_of_several_blocks_a_warp(A, offset, blocks):  # noqa: F811
    fill = Zeros(A, FILL[blocks] + 77, "f32", "f32", 8, offset)
    cases = [Case(A, 200 + n, n, "f32", "f32", 8, offset) for n in COUNTS]
    guarded = [[torch.full((c.count + 64 + offset,), 7.0, device="cuda") for c in cases] for _ in range(2)]
    out = [[t[32 + offset:32 + offset + c.count] for t, c in zip(ts, cases)] + [torch.ones(offset + fill.m.numel(), device="cuda")[offset:]]
           for ts in guarded]
    A.adamw_values([c.m for c in cases] + [fill.m], [c.v for c in cases] + [fill.v], [c.scales for c in cases] + [fill.scales], out=out)
    for i, c in enumerate(cases):
        for got, want, full in zip((out[0][i], out[1][i]), c.state(), (guarded[0][i], guarded[1][i])):
            assert np.array_equal(values(got), want), c.count
            got.fill_(7.0)
            assert (full == 7.0).all(), c.count
    assert not out[0][-1].any() and not out[1][-1].any()
