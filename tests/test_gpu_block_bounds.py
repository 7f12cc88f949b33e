"""GPU tests of what the operators around the banks write: every result inside its view and
nothing beside it.  The results are views of wider buffers, filled with a value whose survival
around the view is checked; the values inside have the bars of test_gpu_block_ops.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, DT, act_ref, close, linear_grad_check, make_weight, randn  # noqa: E402,F401  (A: fixture)

GUARD = 7.0


class Guarded:
    """A view [rows, width] that starts `offset` elements into rows of `pitch`, guard rows around it."""

    def __init__(self, rows, width, dtype, pitch, offset):
        self.buf = torch.full((rows + 4, pitch), GUARD, device="cuda", dtype=DT[dtype])
        self.view = self.buf[2:2 + rows, offset:offset + width]

    def untouched_around(self):
        self.view.fill_(GUARD)
        return bool((self.buf == GUARD).all())


def pitches(width, dtype):
    """(pitch, offset): rows on 16-byte boundaries whose width may end inside 16 bytes, and two off them."""
    unit = 16 // DT[dtype].itemsize
    whole = -(-width // unit) * unit
    return [(whole + unit, 0), (whole + 2 * unit, unit), (width + 1, 0), (whole + unit + 1, 1)]


WIDTHS = [1, 2, 63, 65, 97, 100, 103, 104, 129, 255, 771, 2815]


def native_linear(A, x, w, b, act, res, y, z):  # noqa: F811
    """The C call, which takes a strided z (the Python call allocates its own)."""
    import ctypes
    tr = w.stride(1) != 1
    d = A.LinearDesc(x.data_ptr(), w.data_ptr(), b.data_ptr(), res.data_ptr() if res is not None else 0, y.data_ptr(),
                     z.data_ptr(), x.shape[0], x.stride(0), w.stride(1) if tr else w.stride(0),
                     res.stride(0) if res is not None else 0, y.stride(0), z.stride(0), w.shape[0], w.shape[1],
                     1 if x.dtype == torch.bfloat16 else 2, 0, A.ACTIVATIONS[act], int(tr))
    lib = A.library()
    need = lib.anvil_linear_workspace_bytes(d)
    ws = torch.empty(max(need, 1), device="cuda", dtype=torch.uint8)
    assert lib.anvil_linear_forward(d, ws.data_ptr(), need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == A.OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,k", [(1, 96), (2, 520), (40, 96), (300, 96), (300, 832), (2000, 64)])
def test_linear_forward_writes_its_view(A, rows, k, dtype):  # noqa: F811
    for i, n in enumerate(WIDTHS):
        for j, (pitch, offset) in enumerate(pitches(n, dtype)):
            x, w = randn(1, rows, k, dtype=dtype), make_weight(2, n, k, dtype, (i + j) % 2 == 1)
            b = randn(3, n)
            res = Guarded(rows, n, dtype, pitch, offset).view if j % 2 else None
            y, z = Guarded(rows, n, dtype, pitch, offset), Guarded(rows, n, dtype, *pitches(n, dtype)[(j + 1) % 4])
            native_linear(A, x, w, b, "relu", res, y.view, z.view)
            zr = x.double() @ w.double().t() + b.double()
            mag, c = x.double().abs() @ w.double().abs().t() + b.double().abs(), 2 * (k / 16 + 4)
            close(z.view, zr, dtype, mag, c, ("z", n, pitch, offset))
            more = GUARD if res is not None else 0.0
            close(y.view, act_ref(zr, "relu") + more, dtype, mag + more, c, ("y", n, pitch, offset))
            assert y.untouched_around() and z.untouched_around(), (n, pitch, offset)
            plain = Guarded(rows, n, dtype, pitch, offset)
            A.linear_forward(x, w, out=plain.view)
            close(plain.view, zr - b.double(), dtype, mag, c, ("plain", n, pitch, offset))
            assert plain.untouched_around(), (n, pitch, offset)
    assert A.device_error() == A.OK


def native_linear_backward(A, dy, x, w, dx, dw):  # noqa: F811
    """The C call, which takes a strided dx; w by rows."""
    import ctypes
    code = 1 if x.dtype == torch.bfloat16 else 2
    d = A.LinearGradDesc(dy.data_ptr(), x.data_ptr(), w.data_ptr(), 0, dx.data_ptr(), dw.data_ptr(), 0, x.shape[0],
                         dy.stride(0), x.stride(0), w.stride(0), 0, dx.stride(0), dw.stride(0), w.shape[0], w.shape[1], code,
                         0 if dw.dtype == torch.float32 else code, 0, 0, 0)
    lib = A.library()
    need = lib.anvil_linear_backward_workspace_bytes(d)
    ws = torch.empty(max(need, 1), device="cuda", dtype=torch.uint8)
    assert lib.anvil_linear_backward(d, ws.data_ptr(), need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == A.OK


@pytest.mark.parametrize("dw_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(3, 96), (300, 72), (300, 1), (5000, 200)])
def test_linear_backward_writes_its_views(A, rows, n, dw_type):  # noqa: F811
    for k in WIDTHS:
        for j in range(4):
            dy, x = randn(1, rows, n, dtype="bf16"), randn(2, rows, k, dtype="bf16")
            w = randn(3, n, k, dtype="bf16", scale=k ** -0.5)
            dx = Guarded(rows, k, "bf16", *pitches(k, "bf16")[j])
            dw = Guarded(n, k, dw_type, *pitches(k, dw_type)[(j + 1) % 4])
            native_linear_backward(A, dy, x, w, dx.view, dw.view)
            linear_grad_check(A, dy, x, w, None, None, "bf16", dw_type, (dx.view, dw.view, None))
            assert dx.untouched_around() and dw.untouched_around(), (k, j)
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dw_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 300])
def test_linear_dweight_by_columns_writes_its_view(A, rows, dw_type):  # noqa: F811
    k = 136
    for n in WIDTHS[1:]:
        for pitch, offset in pitches(n, dw_type):
            dy, x = randn(1, rows, n, dtype="bf16"), randn(2, rows, k, dtype="bf16")
            w = make_weight(3, n, k, "bf16", True)
            dw = Guarded(k, n, dw_type, pitch, offset)
            got = A.linear_backward(dy, x, w, dweight=dw.view.t(), need_dx=False, bias_grad=False)
            linear_grad_check(A, dy, x, w, None, None, "bf16", dw_type, got)
            assert dw.untouched_around(), (n, pitch, offset)
    assert A.device_error() == A.OK


def stored(kind, n, k, dtype, fill):
    """A view [n, k] of a larger buffer, both filled with `fill` (a value, or a function of a shape):
    (buffer, view)."""
    if kind == "rows":            # contiguous rows, guard rows before and after
        buf = fill((n + 4, k)).to(DT[dtype])
        return buf, buf[2:2 + n]
    if kind == "wide rows":       # rows of a wider buffer
        buf = fill((n + 4, k + 9)).to(DT[dtype])
        return buf, buf[2:2 + n, 8:8 + k]
    if kind == "columns":         # the transpose of contiguous rows
        buf = fill((k + 4, n)).to(DT[dtype])
        return buf, buf[2:2 + k].t()
    buf = fill((k + 4, n + 9)).to(DT[dtype])  # "wide columns"
    return buf, buf[2:2 + k, 8:8 + n].t()


KINDS = ("rows", "wide rows", "columns", "wide columns")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("shape", [(1, 1), (1, 96), (1, 515), (96, 1), (515, 1), (72, 96), (33, 65)], ids=lambda s: "x".join(map(str, s)))
def test_dweight_in_its_own_place(A, shape, rows, accumulate):  # noqa: F811
    """Every storage of weight with every storage of the caller's dweight: the gradient lands in the
    view and nowhere else, or (orders that differ, more than one row and column) is refused."""
    n, k = shape
    dy, x = randn(1, rows, n, dtype="bf16"), randn(2, rows, k, dtype="bf16")
    dense = randn(3, n, k, dtype="bf16", scale=k ** -0.5)
    for wk in KINDS:
        _, w = stored(wk, n, k, "bf16", lambda s: torch.zeros(s, device="cuda"))
        w.copy_(dense)
        for gk in KINDS:
            for dw_type in ("f32", "bf16"):
                buf, view = stored(gk, n, k, dw_type, lambda s: torch.full(s, 7.0, device="cuda"))
                before = buf.clone()
                db = torch.full((n,), 5.0, device="cuda")
                if n > 1 and k > 1 and wk.split()[-1] != gk.split()[-1]:
                    with pytest.raises(ValueError, match="shape and order"):
                        A.linear_backward(dy, x, w, dweight=view, dbias=db, accumulate=accumulate)
                    assert torch.equal(buf, before)
                    continue
                dx, dw, db = A.linear_backward(dy, x, w, dweight=view, dbias=db, accumulate=accumulate)
                assert dw.data_ptr() == view.data_ptr() and dw.stride() == view.stride()
                want = A.linear_backward(dy, x, dense, dweight_dtype=DT[dw_type])
                if accumulate:
                    full = torch.full((n, k), 7.0, device="cuda").to(DT[dw_type])
                    want = A.linear_backward(dy, x, dense, dweight=full, dbias=torch.full((n,), 5.0, device="cuda"),
                                             accumulate=True)
                    p, mag = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
                    u = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}[dw_type]
                    # as for the products without it: 2 E per 16 rows, one rounding of the sum
                    bar = u * (p + 7).abs() + (2 * (rows / 16 + 4) + 8) * 2.0 ** -24 * (mag + 7)
                    assert ((want[1].double() - p - 7).abs() <= bar).all()
                else:
                    linear_grad_check(A, dy, x, dense, None, None, "bf16", dw_type, want)
                # another order of the operands may add up in another order: one rounding each
                tol = {"f32": 2.0 ** -20, "bf16": 2.0 ** -7}[dw_type]
                scale = dy.double().abs().t() @ x.double().abs() + (7 if accumulate else 0)
                assert ((dw.double() - want[1].double()).abs() <= tol * scale).all(), (wk, gk)
                dxs = dy.double().abs() @ dense.double().abs()
                assert ((dx.double() - want[0].double()).abs() <= 2.0 ** -7 * dxs).all()
                assert torch.equal(db, want[2])
                view.fill_(7.0)
                assert torch.equal(buf, before), (wk, gk, dw_type)
    assert A.device_error() == A.OK


def padded(seed, rows, width, dtype, pitch, offset):
    """Normal values in a view of wider rows whose other elements are NaN."""
    buf = torch.full((rows, pitch), float("nan"), device="cuda", dtype=DT[dtype])
    view = buf[:, offset:offset + width]
    view.copy_(randn(seed, rows, width, dtype=dtype))
    return view


# narrow and wide teams, and rows enough for the kernels that keep several rows on their way
NORM_VIEWS = [(1, 7), (37, 63), (300, 255), (9, 1023), (300, 1024), (41, 2815), (3, 5001), (2, 9999), (2, 16384),
              (20001, 300), (14801, 1023), (29301, 1024), (14701, 2815), (14701, 2816)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", NORM_VIEWS, ids=lambda s: "x".join(map(str, s)))
def test_norm_writes_its_views(A, shape, dtype):  # noqa: F811
    """The same results as from contiguous copies, to the last rounding, and nothing beside them."""
    rows, n = shape
    w, b = 1 + randn(3, n, scale=0.2), randn(4, n, scale=0.2)
    u = {"f32": 2.0 ** -18, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]  # sums of another order, one rounding each
    for j, (pitch, offset) in enumerate(pitches(n, dtype)):
        other = pitches(n, dtype)[(j + 2) % 4]
        x, dy, res = padded(5, rows, n, dtype, pitch, offset), padded(6, rows, n, dtype, *other), padded(7, rows, n, dtype, pitch, offset)
        y, dx = Guarded(rows, n, dtype, pitch, offset), Guarded(rows, n, dtype, *other)
        _, mean, rstd = A.layernorm_forward(x, w, b, out=y.view)
        wy, wm, wr = A.layernorm_forward(x.contiguous(), w, b)
        with_res = res if j % 2 else None
        _, dw, db = A.layernorm_backward(dy, x, wm, wr, w, residual_grad=with_res, out=dx.view)
        want = A.layernorm_backward(dy.contiguous(), x.contiguous(), wm, wr, w,
                                    residual_grad=with_res.contiguous() if j % 2 else None)
        # y: the mean's and the variance's order of addition; a value of 0 has that of its terms
        assert ((y.view.double() - wy.double()).abs() <= u * (wy.double().abs() + 1)).all()
        assert torch.allclose(mean, wm, atol=1e-5, rtol=0) and torch.allclose(rstd, wr, rtol=1e-5, atol=0)
        assert ((dx.view.double() - want[0].double()).abs() <= u * (want[0].double().abs() + wr.double()[:, None] * 4 + 1)).all()
        # sqrt(rows) of the terms' size, and the rounding of their sums
        assert torch.allclose(dw, want[1], rtol=1e-4, atol=2e-5 * rows ** 0.5 + 1e-5)
        assert torch.allclose(db, want[2], rtol=1e-4, atol=2e-5 * rows ** 0.5 + 1e-5)
        assert y.untouched_around() and dx.untouched_around(), (pitch, offset)
    assert A.device_error() == A.OK


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 129), (5, 5003), (160, 4099), (1, 50257)], ids=lambda s: "x".join(map(str, s)))
def test_logprob_writes_its_view(A, shape, dtype):  # noqa: F811
    rows, vocab = shape
    t = torch.arange(rows, device="cuda") * 37 % vocab
    gl, gh = randn(1, rows), randn(2, rows)
    for j, (pitch, offset) in enumerate(pitches(vocab, dtype)):
        x = padded(3, rows, vocab, dtype, pitch, offset)
        top = min(vocab, 9)
        got, want = A.token_logprobs(x, t, top=top), A.token_logprobs(x.contiguous(), t, top=top)
        assert torch.equal(got[4], want[4])
        for p, q in zip(got[:4], want[:4]):  # sums of another order: at most 30 in magnitude, 192 roundings
            assert torch.allclose(p, q, rtol=0, atol=30 * 192 * 2.0 ** -24)
        d = Guarded(rows, vocab, dtype, *pitches(vocab, dtype)[(j + j // 2) % 4])
        A.token_logprobs_backward(x, t, want[2], gl, entropy=want[1], grad_entropy=gh, out=d.view)
        ref = A.token_logprobs_backward(x.contiguous(), t, want[2], gl, entropy=want[1], grad_entropy=gh)
        u = {"f32": 2.0 ** -18, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
        assert ((d.view.double() - ref.double()).abs() <= u * ref.double().abs() + 2.0 ** -23).all()
        assert d.untouched_around(), (pitch, offset)
    assert A.device_error() == A.OK


def test_offsets_past_32_bits_backward_and_results(A):  # noqa: F811
    """Every array of the backward passes, and the results, as rows 2^28 elements apart."""
    ld, rows, n = 1 << 28, 10, 768

    def far(seed, width, dtype=torch.bfloat16, scale=1.0):
        buf = torch.empty(ld * (rows - 1) + width, dtype=dtype, device="cuda")
        view = torch.as_strided(buf, (rows, width), (ld, 1))
        if seed is not None:
            view.copy_(randn(seed, rows, width, scale=scale))
        return view
    x, dy, out = far(1, n), far(2, n), far(None, n)
    y, mean, rstd = A.layernorm_forward(x, out=out)
    assert torch.equal(y, A.layernorm_forward(x.contiguous())[0])
    got = A.layernorm_backward(dy, x, mean, rstd, residual_grad=dy, out=out)
    want = A.layernorm_backward(dy.contiguous(), x.contiguous(), mean, rstd, residual_grad=dy.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    w = randn(3, n, n, dtype="bf16", scale=n ** -0.5)
    assert torch.equal(A.linear_forward(x, w, residual=dy, out=out),
                       A.linear_forward(x.contiguous(), w, residual=dy.contiguous()))
    dw = torch.empty((n, n), device="cuda")
    native_linear_backward(A, dy, x, w, out, dw)
    rdx, rdw, _ = A.linear_backward(dy.contiguous(), x.contiguous(), w, bias_grad=False, dweight_dtype=torch.float32)
    assert torch.equal(out, rdx) and torch.equal(dw, rdw)
    del x, dy, out, got, y
    # a weight and its gradient whose rows are that far apart
    w, dw = far(4, 264, scale=0.1), far(None, 264, torch.float32)
    x, dy = randn(5, 300, 264, dtype="bf16"), randn(6, 300, rows, dtype="bf16")
    dx, _, _ = A.linear_backward(dy, x, w, dweight=dw, bias_grad=False)
    rdx, rdw, _ = A.linear_backward(dy, x, w.contiguous(), bias_grad=False, dweight_dtype=torch.float32)
    assert torch.equal(dx, rdx) and torch.equal(dw, rdw)
    dlogits = A.token_logprobs_backward(w, torch.arange(rows, device="cuda"), randn(7, rows), randn(8, rows),
                                        out=far(None, 264))
    assert torch.equal(dlogits, A.token_logprobs_backward(w.contiguous(), torch.arange(rows, device="cuda"), randn(7, rows),
                                                          randn(8, rows)))
    assert A.device_error() == A.OK


def test_linear_bias_of_the_call_before(A):  # noqa: F811
    """A bias (and residual) that the preceding call made, for products in one piece and in parts."""
    for rows, n, k in ((1000, 2815, 771), (300, 768, 4096), (513, 1000, 2048), (8192, 2816, 768), (3, 2816, 768)):
        x, w = randn(1, rows, k, dtype="bf16"), randn(2, n, k, dtype="bf16", scale=k ** -0.5)
        to_bias = randn(3, n, 4096, dtype="bf16", scale=4096 ** -0.5)
        to_res = randn(4, n, 64, dtype="bf16", scale=0.125)
        plain = A.linear_forward(x, w).double()
        mag = x.double().abs() @ w.double().abs().t()
        bias = torch.empty((1, n), device="cuda", dtype=torch.bfloat16)
        res = torch.empty((rows, n), device="cuda", dtype=torch.bfloat16)
        for step in range(6):
            c, r = randn(10 + step, 1, 4096, dtype="bf16", scale=3.0), randn(20 + step, rows, 64, dtype="bf16")
            A.linear_forward(r, to_res, out=res)
            A.linear_forward(c, to_bias, out=bias)
            y = A.linear_forward(x, w, bias[0], residual=res)
            want = plain + bias.double() + res.double()
            # plain is rounded once itself; the products of the two calls may be split differently
            close(y, want, "bf16", 2.0 ** 16 * plain.abs() + mag + bias.double().abs() + res.double().abs(), 4 * (k / 16 + 4), step)
    assert A.device_error() == A.OK
