"""Host-side checks of the operators around the banks that need no GPU: every bad argument
is refused with the documented status before any CUDA call (the pointers are fake), the
workspace sizes, and the Python binding's refusals."""
import pytest

anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")
L = anvil.library()
G = 1 << 36  # fake, aligned device addresses far apart


def fill(cls, base, kw):
    base.update(kw)
    return cls(*[base[k] for k, _ in cls._fields_])


def norm(**kw):
    d = fill(anvil.LayernormDesc, dict(x=G, weight=2 * G, bias=3 * G, y=4 * G, mean=5 * G, rstd=6 * G, rows=10, ldx=64,
                                       ldy=64, width=64, dtype=1, weight_dtype=0, eps=1e-5), kw)
    return L.anvil_layernorm_forward(d, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), anvil.ERR_INVALID_ARG), (dict(y=0), anvil.ERR_INVALID_ARG), (dict(rows=-1), anvil.ERR_INVALID_ARG),
    (dict(width=0), anvil.ERR_INVALID_ARG), (dict(dtype=3), anvil.ERR_INVALID_ARG), (dict(dtype=-1), anvil.ERR_INVALID_ARG),
    (dict(weight_dtype=2), anvil.ERR_INVALID_ARG), (dict(ldx=63), anvil.ERR_INVALID_ARG),
    (dict(ldy=0), anvil.ERR_INVALID_ARG), (dict(width=16385, ldx=16385, ldy=16385), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(rows=(1 << 30) + 1), anvil.ERR_UNSUPPORTED_SHAPE), (dict(x=G + 1), anvil.ERR_ALIGNMENT),
    (dict(weight=2 * G + 2), anvil.ERR_ALIGNMENT), (dict(mean=5 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(y=G + 128), anvil.ERR_ALIAS),              # y over x, shifted by a row
    (dict(y=G, ldy=128), anvil.ERR_ALIAS),           # the same start, another stride
    (dict(mean=4 * G + 64), anvil.ERR_ALIAS), (dict(rstd=5 * G), anvil.ERR_ALIAS), (dict(y=2 * G), anvil.ERR_ALIAS),
    (dict(x=G, ldx=128, y=G + 126, ldy=128), anvil.ERR_ALIAS),  # interleaved rows one element too close
])
def test_layernorm_forward_refusals(kw, code):
    assert norm(**kw) == code


def norm_grad(ws=1 << 50, wsb=1 << 40, **kw):
    d = fill(anvil.LayernormGradDesc, dict(dy=G, x=2 * G, mean=3 * G, rstd=4 * G, weight=5 * G, residual_grad=6 * G,
                                           dx=7 * G, dweight=8 * G, dbias=9 * G, rows=1000, lddy=64, ldx=64, ldr=64,
                                           lddx=64, width=64, dtype=1, weight_dtype=0), kw)
    return L.anvil_layernorm_backward(d, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), anvil.ERR_INVALID_ARG), (dict(x=0), anvil.ERR_INVALID_ARG), (dict(mean=0), anvil.ERR_INVALID_ARG),
    (dict(rstd=0), anvil.ERR_INVALID_ARG), (dict(ldr=1), anvil.ERR_INVALID_ARG), (dict(lddx=1), anvil.ERR_INVALID_ARG),
    (dict(dweight=8 * G + 2), anvil.ERR_ALIGNMENT), (dict(dx=G + 2), anvil.ERR_ALIAS), (dict(dx=G, lddx=65), anvil.ERR_ALIAS),
    (dict(dbias=8 * G), anvil.ERR_ALIAS), (dict(dweight=7 * G), anvil.ERR_ALIAS), (dict(dx=5 * G), anvil.ERR_ALIAS),
    (dict(ws=0), anvil.ERR_WORKSPACE), (dict(wsb=16), anvil.ERR_WORKSPACE), (dict(ws=(1 << 50) + 16), anvil.ERR_ALIGNMENT),
    (dict(ws=2 * G), anvil.ERR_ALIAS),
])
def test_layernorm_backward_refusals(kw, code):
    assert norm_grad(**kw) == code


def linear(ws=1 << 50, wsb=1 << 40, **kw):
    d = fill(anvil.LinearDesc, dict(x=G, weight=2 * G, bias=3 * G, residual=4 * G, y=5 * G, preact=6 * G, rows=100, ldx=64,
                                    ldw=64, ldr=96, ldy=96, ldz=96, n=96, k=64, dtype=1, bias_dtype=0, activation=2,
                                    weight_transposed=0), kw)
    return L.anvil_linear_forward(d, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), anvil.ERR_INVALID_ARG), (dict(weight=0), anvil.ERR_INVALID_ARG), (dict(y=0), anvil.ERR_INVALID_ARG),
    (dict(dtype=0), anvil.ERR_INVALID_ARG), (dict(bias_dtype=2), anvil.ERR_INVALID_ARG),
    (dict(activation=6), anvil.ERR_INVALID_ARG), (dict(activation=-1), anvil.ERR_INVALID_ARG),
    (dict(n=0), anvil.ERR_INVALID_ARG), (dict(k=0), anvil.ERR_INVALID_ARG), (dict(rows=-1), anvil.ERR_INVALID_ARG),
    (dict(ldw=63), anvil.ERR_INVALID_ARG), (dict(weight_transposed=1), anvil.ERR_INVALID_ARG),  # ldw < n
    (dict(ldy=95), anvil.ERR_INVALID_ARG), (dict(ldr=95), anvil.ERR_INVALID_ARG), (dict(ldz=95), anvil.ERR_INVALID_ARG),
    (dict(n=(1 << 20) + 1, ldy=1 << 21, ldr=1 << 21, ldz=1 << 21), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(x=G + 1), anvil.ERR_ALIGNMENT), (dict(bias=3 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(y=G), anvil.ERR_ALIAS), (dict(y=4 * G + 2), anvil.ERR_ALIAS), (dict(preact=4 * G), anvil.ERR_ALIAS),
    (dict(preact=5 * G + 64), anvil.ERR_ALIAS), (dict(y=2 * G + 96), anvil.ERR_ALIAS),
    # an operand off its 16-byte boundary needs a copy, so a workspace
    (dict(x=G + 2, ws=0), anvil.ERR_WORKSPACE), (dict(x=G + 2, wsb=100), anvil.ERR_WORKSPACE),
    (dict(x=G + 2, ws=(1 << 50) + 8), anvil.ERR_ALIGNMENT), (dict(x=G + 2, ws=5 * G), anvil.ERR_ALIAS),
])
def test_linear_forward_refusals(kw, code):
    assert linear(**kw) == code


def linear_grad_desc(**kw):
    return fill(anvil.LinearGradDesc, dict(dy=G, x=2 * G, weight=3 * G, preact=4 * G, dx=5 * G, dweight=6 * G, dbias=7 * G,
                                           rows=100, lddy=96, ldx=64, ldw=64, ldz=96, lddx=64, lddw=64, n=96, k=64, dtype=1,
                                           dweight_dtype=0, activation=2, weight_transposed=0, accumulate=0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), anvil.ERR_INVALID_ARG), (dict(x=0), anvil.ERR_INVALID_ARG), (dict(weight=0), anvil.ERR_INVALID_ARG),
    (dict(preact=0), anvil.ERR_INVALID_ARG), (dict(dweight_dtype=2), anvil.ERR_INVALID_ARG),
    (dict(dtype=0), anvil.ERR_INVALID_ARG), (dict(lddw=63), anvil.ERR_INVALID_ARG), (dict(ldz=95), anvil.ERR_INVALID_ARG),
    (dict(lddx=63), anvil.ERR_INVALID_ARG), (dict(dweight=6 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(dbias=7 * G + 2), anvil.ERR_ALIGNMENT), (dict(dx=2 * G), anvil.ERR_ALIAS), (dict(dx=G), anvil.ERR_ALIAS),
    (dict(dweight=3 * G), anvil.ERR_ALIAS), (dict(dbias=6 * G), anvil.ERR_ALIAS), (dict(dx=4 * G), anvil.ERR_ALIAS),
    (dict(ws=0), anvil.ERR_WORKSPACE), (dict(wsb=64), anvil.ERR_WORKSPACE), (dict(ws=(1 << 50) + 64), anvil.ERR_ALIGNMENT),
    (dict(ws=6 * G), anvil.ERR_ALIAS),
])
def test_linear_backward_refusals(kw, code):
    ws, wsb = kw.pop("ws", 1 << 50), kw.pop("wsb", 1 << 40)
    assert L.anvil_linear_backward(linear_grad_desc(**kw), ws, wsb, None) == code


def test_linear_workspaces():
    def need(**kw):
        base = dict(x=G, weight=2 * G, bias=0, residual=0, y=5 * G, preact=0, rows=100, ldx=64, ldw=64, ldr=0, ldy=96,
                    ldz=0, n=96, k=64, dtype=1, bias_dtype=0, activation=0, weight_transposed=0)
        return L.anvil_linear_workspace_bytes(fill(anvil.LinearDesc, base, kw))
    assert need() == 0                                  # everything on 16-byte rows
    assert need(x=G + 2) == 100 * 64 * 2                # a copy of x
    assert need(ldx=65, k=64) == 100 * 64 * 2
    assert need(k=63, ldx=63, ldw=63) >= 2 * 64 * (100 + 96)
    assert need(rows=0, x=G + 2) == 0 and need(n=0) == 0
    # dz (an activation), the bias's partial sums; without an activation neither dz nor a copy
    full = L.anvil_linear_backward_workspace_bytes(linear_grad_desc())
    none = L.anvil_linear_backward_workspace_bytes(linear_grad_desc(activation=0, dbias=0))
    assert full >= 100 * 96 * 2 + 4 * 96 and none == 0


def logprob(**kw):
    d = fill(anvil.LogprobDesc, dict(logits=G, targets=2 * G, logprob=3 * G, entropy=4 * G, lse=5 * G, top_logprob=6 * G,
                                     top_index=7 * G, rows=10, ld=100, vocab=100, top=4, dtype=1, targets_int64=1), kw)
    return L.anvil_token_logprobs(d, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=0), anvil.ERR_INVALID_ARG), (dict(targets=0), anvil.ERR_INVALID_ARG), (dict(vocab=0), anvil.ERR_INVALID_ARG),
    (dict(top=33), anvil.ERR_INVALID_ARG), (dict(top=-1), anvil.ERR_INVALID_ARG), (dict(vocab=3, top=4), anvil.ERR_INVALID_ARG),
    (dict(top_index=0), anvil.ERR_INVALID_ARG), (dict(top_logprob=0), anvil.ERR_INVALID_ARG), (dict(ld=99), anvil.ERR_INVALID_ARG),
    (dict(dtype=7), anvil.ERR_INVALID_ARG), (dict(vocab=1 << 25, ld=1 << 25), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(logits=G + 1), anvil.ERR_ALIGNMENT), (dict(targets=2 * G + 4), anvil.ERR_ALIGNMENT),
    (dict(lse=3 * G), anvil.ERR_ALIAS), (dict(entropy=G + 4), anvil.ERR_ALIAS), (dict(top_index=6 * G + 16), anvil.ERR_ALIAS),
])
def test_token_logprobs_refusals(kw, code):
    assert logprob(**kw) == code


def logprob_grad(**kw):
    d = fill(anvil.LogprobGradDesc, dict(logits=G, targets=2 * G, lse=3 * G, entropy=4 * G, grad_logprob=5 * G,
                                         grad_entropy=6 * G, dlogits=7 * G, rows=10, ld=100, ldd=100, vocab=100, dtype=1,
                                         targets_int64=0), kw)
    return L.anvil_token_logprobs_backward(d, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=0), anvil.ERR_INVALID_ARG), (dict(lse=0), anvil.ERR_INVALID_ARG), (dict(targets=0), anvil.ERR_INVALID_ARG),
    (dict(entropy=0), anvil.ERR_INVALID_ARG), (dict(ldd=99), anvil.ERR_INVALID_ARG),
    (dict(rows=1 << 30, vocab=1 << 20, ld=1 << 20, ldd=1 << 20), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(dlogits=7 * G + 1), anvil.ERR_ALIGNMENT), (dict(dlogits=G + 2), anvil.ERR_ALIAS),
    (dict(dlogits=3 * G), anvil.ERR_ALIAS), (dict(dlogits=G, ldd=104), anvil.ERR_ALIAS),
])
def test_token_logprobs_backward_refusals(kw, code):
    assert logprob_grad(**kw) == code


def test_no_rows_is_no_work():
    """Forward calls and gradients of inputs over no rows return before any CUDA call."""
    assert norm(rows=0) == linear(rows=0) == logprob(rows=0) == logprob_grad(rows=0) == anvil.OK
    assert norm_grad(rows=0, dweight=0, dbias=0) == anvil.OK
    assert L.anvil_linear_backward(linear_grad_desc(rows=0, accumulate=1), 0, 0, None) == anvil.OK


def test_null_descriptors():
    for f in (L.anvil_layernorm_forward, L.anvil_token_logprobs, L.anvil_token_logprobs_backward):
        assert f(None, None) == anvil.ERR_INVALID_ARG
    for f in (L.anvil_layernorm_backward, L.anvil_linear_forward, L.anvil_linear_backward):
        assert f(None, None, 0, None) == anvil.ERR_INVALID_ARG
    for f in (L.anvil_linear_workspace_bytes, L.anvil_linear_backward_workspace_bytes,
              L.anvil_layernorm_backward_workspace_bytes):
        assert f(None) == 0


def test_structures_match_the_header():
    """Field names and order of each descriptor are those of the header's struct."""
    import re
    text = re.sub(r"/\*.*?\*/", "", open(anvil.HEADER).read(), flags=re.S)
    for cls, name in ((anvil.LayernormDesc, "anvil_layernorm_desc"), (anvil.LayernormGradDesc, "anvil_layernorm_grad_desc"),
                      (anvil.LinearDesc, "anvil_linear_desc"), (anvil.LinearGradDesc, "anvil_linear_grad_desc"),
                      (anvil.LogprobDesc, "anvil_logprob_desc"), (anvil.LogprobGradDesc, "anvil_logprob_grad_desc")):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
        fields = [f for decl in body.split(";") for f in re.findall(r"(\w+)\s*(?:,|$)", decl.strip())]
        assert fields == [f for f, _ in cls._fields_], name


def test_binding_refusals():
    import torch
    bf = torch.bfloat16
    x, w = torch.zeros((4, 8), dtype=bf), torch.zeros((6, 8), dtype=bf)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.layernorm_forward(x)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.linear_forward(x, w)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
        anvil.layernorm_forward(x.double())
    with pytest.raises(ValueError, match="rows must be contiguous"):
        anvil.layernorm_forward(x.t())
    with pytest.raises(ValueError, match="rows overlap"):
        anvil.layernorm_forward(x[0].expand(5, 8))
    with pytest.raises(ValueError, match="common row stride"):
        anvil.layernorm_forward(torch.zeros((3, 4, 8))[:, ::3])
    with pytest.raises(ValueError, match="vector of 8"):
        anvil.layernorm_forward(x, torch.zeros(7))
    with pytest.raises(ValueError, match="fp32 or of x's type"):
        anvil.layernorm_forward(x, torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError, match="dy must have"):
        anvil.layernorm_backward(x[:2], x, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="mean must be"):
        anvil.layernorm_backward(x, x, torch.zeros(3), torch.zeros(4))
    with pytest.raises(ValueError, match="bf16 or fp16"):
        anvil.linear_forward(x.float(), w.float())
    with pytest.raises(ValueError, match=r"\[n, 8\]"):
        anvil.linear_forward(x, torch.zeros((6, 9), dtype=bf))
    with pytest.raises(ValueError, match=r"must be \[n, k\]"):
        anvil.linear_forward(x, w.half())
    with pytest.raises(ValueError, match="by rows or by columns"):
        anvil.linear_forward(x, torch.zeros((6, 16), dtype=bf)[:, ::2])
    with pytest.raises(ValueError, match="activation must be"):
        anvil.linear_forward(x, w, activation="swish")
    with pytest.raises(ValueError, match="residual must have"):
        anvil.linear_forward(x, w, residual=x)
    with pytest.raises(ValueError, match="preact is needed"):
        anvil.linear_backward(torch.zeros((4, 6), dtype=bf), x, w, activation="gelu")
    with pytest.raises(ValueError, match="accumulate needs"):
        anvil.linear_backward(torch.zeros((4, 6), dtype=bf), x, w, accumulate=True)
    with pytest.raises(ValueError, match="dweight must be fp32"):
        anvil.linear_backward(torch.zeros((4, 6), dtype=bf), x, w, dweight_dtype=torch.float16)
    with pytest.raises(ValueError, match="top must be"):
        anvil.token_logprobs(x, top=9)
    with pytest.raises(ValueError, match="targets must be"):
        anvil.token_logprobs(x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="grad_entropy needs"):
        anvil.token_logprobs_backward(x, None, torch.zeros(4), grad_entropy=torch.zeros(4))
    with pytest.raises(ValueError, match="grad_logprob needs"):
        anvil.token_logprobs_backward(x, None, torch.zeros(4), torch.zeros(4))
