"""The linear layer's gradient with dz in two parts: refusals and workspaces (no GPU needed), and on a
GPU bars that one rounding of dz to 16 bits exceeds."""
import pytest

torch = pytest.importorskip("torch")
anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")

from test_block_abi import L, linear_grad_desc  # noqa: E402

TWO = 256  # ANVIL_DZ_TWO_PARTS


def test_the_headers_code():
    import re
    assert int(re.search(r"#define ANVIL_DZ_TWO_PARTS (\d+)", open(anvil.HEADER).read()).group(1)) == TWO


@pytest.mark.parametrize("kw,code", [
    (dict(activation=TWO + 6), anvil.ERR_INVALID_ARG), (dict(activation=2 * TWO), anvil.ERR_INVALID_ARG),
    (dict(activation=TWO + 2, preact=0), anvil.ERR_INVALID_ARG),
    (dict(activation=TWO + 2, rows=(1 << 29) + 1), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(activation=TWO + 2, wsb=1000), anvil.ERR_WORKSPACE),
])
def test_refusals(kw, code):
    wsb = kw.pop("wsb", 1 << 40)
    assert L.anvil_linear_backward(linear_grad_desc(**kw), 1 << 50, wsb, None) == code


def test_workspaces():
    need = lambda **kw: L.anvil_linear_backward_workspace_bytes(linear_grad_desc(**kw))  # noqa: E731
    # without an activation there is nothing to keep; with one, dz, x and the weight twice
    assert need(activation=TWO, dbias=0) == need(activation=0, dbias=0) == 0
    assert need(activation=TWO + 2) >= need(activation=2) + 2 * (100 * 96 + 2 * 100 * 64 + 2 * 96 * 64)
    assert need(activation=TWO + 2, dx=0, dweight=0) == need(activation=2, dx=0, dweight=0)


def test_binding_refuses():
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dz_parts must be 1 or 2"):
        anvil.linear_backward(t, t, t, dz_parts=3)


SHAPES = [(1, 1, 1), (1, 2816, 768), (2, 65, 7), (3, 300, 129), (17, 100, 1000), (64, 768, 768), (129, 257, 256), (300, 2815, 771),
          (513, 1, 100), (700, 1000, 1), (1000, 768, 2816), (2048, 256, 768), (5000, 200, 264), (9000, 64, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradients(shape, transposed, dtype):
    from test_gpu_block_ops import DT, E, U, act_slope_ref, close, make_weight, randn
    A = anvil
    rows, n, k = shape
    for i, (act, dw_type, pad, off) in enumerate([("relu2", "f32", 0, 0), ("gelu", dtype, 1, 1), ("silu", "f32", 8, 0)]):
        dy, x = randn(1, rows, n, dtype=dtype, pad=pad, offset=off), randn(2, rows, k, dtype=dtype, pad=pad, offset=off)
        w, z = make_weight(3, n, k, dtype, transposed, pad, off), randn(4, rows, n, dtype=dtype, pad=pad)
        dx, dw, db = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=DT[dw_type], dz_parts=2)
        dz = dy.double() * act_slope_ref(z.double(), act)
        # dz's own arithmetic: 16 roundings; its parts: U^2 of it, and the second one's subnormals in fp16
        err = 16 * E * (dy.double().abs() * (2 * z.double().abs() + 2)) + U[dtype] ** 2 * dz.abs() \
            + (2.0 ** -25 if dtype == "f16" else 0.0)
        # the accumulator over twice the contraction: 2 E per 16-deep step; fp32 results by chains of 512
        c = 2 * (2 * (n + 7) / 16 + 4)
        close(dx, dz @ w.double(), dtype, dz.abs() @ w.double().abs() * (1 + U[dtype]) + err @ w.double().abs() / E / c, c, (act, "dx"))
        c = 2 * 36 + 2 * rows / 512 + 8 if dw_type == "f32" else 2 * (2 * rows / 16 + 4)
        close(dw, dz.t() @ x.double(), dw_type, dz.abs().t() @ x.double().abs() * (1 + U[dtype])
              + err.t() @ x.double().abs() / E / c, c, (act, "dweight"))
        want = A.linear_backward(dy, x, w, preact=z, activation=act, need_dx=False, need_dweight=False)[2]
        assert torch.equal(db, want)
        if rows > 100 and dw_type == "f32":  # and one part is not that near
            one = A.linear_backward(dy, x, w, preact=z, activation=act, dweight_dtype=torch.float32)[1]
            ref = dz.t() @ x.double()
            assert float((one.double() - ref).norm()) > 8 * float((dw.double() - ref).norm())
    assert A.device_error() == A.OK


@pytest.mark.gpu
def test_accumulate_subsets_and_no_activation():
    from test_gpu_block_ops import randn
    A = anvil
    dy, x, w, z = (randn(i, *s, dtype="bf16") for i, s in enumerate(((300, 200), (300, 136), (200, 136), (300, 200))))
    kw = dict(preact=z, activation="silu", dz_parts=2, dweight_dtype=torch.float32)
    dx, dw, db = A.linear_backward(dy, x, w, **kw)
    assert torch.equal(A.linear_backward(dy, x, w, need_dweight=False, bias_grad=False, **kw)[0], dx)
    assert torch.equal(A.linear_backward(dy, x, w, need_dx=False, bias_grad=False, **kw)[1], dw)
    assert all(torch.equal(p, q) for p, q in zip(A.linear_backward(dy, x, w, **kw), (dx, dw, db)))
    dw2, db2 = torch.ones_like(dw), torch.ones_like(db)
    A.linear_backward(dy, x, w, dweight=dw2, dbias=db2, accumulate=True, **kw)
    assert torch.allclose(dw2, dw + 1, rtol=1e-6, atol=1e-6) and torch.allclose(db2, db + 1, rtol=1e-6, atol=1e-5)
    # nothing to keep without an activation: the same bits
    assert all(torch.equal(p, q) for p, q in zip(A.linear_backward(dy, x, w, dz_parts=2), A.linear_backward(dy, x, w)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = A.linear_backward(dy, x, w, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
