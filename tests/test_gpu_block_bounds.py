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
