"""The gated layer, what needs no GPU: refusals before any CUDA call (the pointers are fake), workspace
sizes, the binding's refusals."""
import re

import pytest

anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")
L = anvil.library()
G = 1 << 36  # fake, aligned device addresses far apart


def fill(cls, base, kw):
    base.update(kw)
    return cls(*[base[k] for k, _ in cls._fields_])


def desc(**kw):
    return fill(anvil.GatedDesc, dict(x=G, gate=2 * G, up=3 * G, y=4 * G, preact_gate=5 * G, preact_up=6 * G, rows=100, ldx=64,
                                      ldgate=64, ldup=64, ldy=96, ldzg=96, ldzu=96, n=96, k=64, dtype=1, activation=5,
                                      weight_transposed=0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), anvil.ERR_INVALID_ARG), (dict(gate=0), anvil.ERR_INVALID_ARG), (dict(up=0), anvil.ERR_INVALID_ARG),
    (dict(y=0), anvil.ERR_INVALID_ARG), (dict(dtype=0), anvil.ERR_INVALID_ARG), (dict(activation=6), anvil.ERR_INVALID_ARG),
    (dict(activation=-1), anvil.ERR_INVALID_ARG), (dict(n=0), anvil.ERR_INVALID_ARG), (dict(k=0), anvil.ERR_INVALID_ARG),
    (dict(rows=-1), anvil.ERR_INVALID_ARG), (dict(ldgate=63), anvil.ERR_INVALID_ARG), (dict(ldup=63), anvil.ERR_INVALID_ARG),
    (dict(weight_transposed=1), anvil.ERR_INVALID_ARG), (dict(ldy=95), anvil.ERR_INVALID_ARG),
    (dict(ldzg=95), anvil.ERR_INVALID_ARG), (dict(ldzu=95), anvil.ERR_INVALID_ARG),
    (dict(n=(1 << 20) + 1, ldy=1 << 21, ldzg=1 << 21, ldzu=1 << 21), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(x=G + 1), anvil.ERR_ALIGNMENT), (dict(up=3 * G + 1), anvil.ERR_ALIGNMENT), (dict(preact_up=6 * G + 1), anvil.ERR_ALIGNMENT),
    (dict(y=G), anvil.ERR_ALIAS), (dict(y=2 * G + 2), anvil.ERR_ALIAS), (dict(preact_up=5 * G), anvil.ERR_ALIAS),
    (dict(preact_gate=4 * G + 64), anvil.ERR_ALIAS), (dict(preact_gate=3 * G), anvil.ERR_ALIAS),
    (dict(x=G + 2, ws=0), anvil.ERR_WORKSPACE), (dict(up=3 * G + 2, wsb=100), anvil.ERR_WORKSPACE),
    (dict(gate=2 * G + 2, ws=(1 << 50) + 8), anvil.ERR_ALIGNMENT), (dict(x=G + 2, ws=4 * G), anvil.ERR_ALIAS),
])
def test_forward_refusals(kw, code):
    ws, wsb = kw.pop("ws", 1 << 50), kw.pop("wsb", 1 << 40)
    assert L.anvil_gated_linear_forward(desc(**kw), ws, wsb, None) == code


def grad(**kw):
    return fill(anvil.GatedGradDesc, dict(dy=G, x=2 * G, gate=3 * G, up=4 * G, preact_gate=5 * G, preact_up=6 * G, dx=7 * G,
                                          dgate=8 * G, dup=9 * G, rows=100, lddy=96, ldx=64, ldgate=64, ldup=64, ldzg=96,
                                          ldzu=96, lddx=64, lddgate=64, lddup=64, n=96, k=64, dtype=1, dweight_dtype=0,
                                          activation=5, weight_transposed=0, accumulate=0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), anvil.ERR_INVALID_ARG), (dict(x=0), anvil.ERR_INVALID_ARG), (dict(gate=0), anvil.ERR_INVALID_ARG),
    (dict(up=0), anvil.ERR_INVALID_ARG), (dict(preact_gate=0), anvil.ERR_INVALID_ARG), (dict(preact_up=0), anvil.ERR_INVALID_ARG),
    (dict(dgate=0), anvil.ERR_INVALID_ARG), (dict(dup=0), anvil.ERR_INVALID_ARG), (dict(dweight_dtype=2), anvil.ERR_INVALID_ARG),
    (dict(dtype=0), anvil.ERR_INVALID_ARG), (dict(activation=6), anvil.ERR_INVALID_ARG), (dict(activation=6 | 256), anvil.ERR_INVALID_ARG),
    (dict(lddgate=63), anvil.ERR_INVALID_ARG), (dict(lddup=63), anvil.ERR_INVALID_ARG), (dict(lddx=63), anvil.ERR_INVALID_ARG),
    (dict(ldzg=95), anvil.ERR_INVALID_ARG), (dict(lddy=95), anvil.ERR_INVALID_ARG),
    (dict(rows=(1 << 28) + 1), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(dgate=8 * G + 2), anvil.ERR_ALIGNMENT), (dict(dx=7 * G + 1), anvil.ERR_ALIGNMENT), (dict(preact_gate=5 * G + 1), anvil.ERR_ALIGNMENT),
    (dict(dup=8 * G), anvil.ERR_ALIAS), (dict(dx=2 * G), anvil.ERR_ALIAS), (dict(dx=G), anvil.ERR_ALIAS), (dict(dgate=4 * G), anvil.ERR_ALIAS),
    (dict(dup=6 * G), anvil.ERR_ALIAS), (dict(ws=0), anvil.ERR_WORKSPACE), (dict(wsb=64), anvil.ERR_WORKSPACE),
    (dict(ws=(1 << 50) + 64), anvil.ERR_ALIGNMENT), (dict(ws=9 * G), anvil.ERR_ALIAS),
])
def test_backward_refusals(kw, code):
    ws, wsb = kw.pop("ws", 1 << 50), kw.pop("wsb", 1 << 40)
    assert L.anvil_gated_linear_backward(grad(**kw), ws, wsb, None) == code


def test_workspaces_and_no_work():
    need = lambda **kw: L.anvil_gated_linear_workspace_bytes(desc(**kw))  # noqa: E731
    assert need() == 0 and need(x=G + 2) == 100 * 64 * 2 and need(up=3 * G + 2) == 96 * 64 * 2 and need(rows=0, x=G + 2) == 0
    back = lambda **kw: L.anvil_gated_linear_backward_workspace_bytes(grad(**kw))  # noqa: E731
    assert back() >= 2 * 100 * 96 * 2 and back(activation=5 | 256) >= 4 * 100 * 96 * 2
    assert back(dx=0, dgate=0, dup=0) == 0 and back(rows=0) == 0
    assert L.anvil_gated_linear_forward(desc(rows=0), None, 0, None) == anvil.OK
    assert L.anvil_gated_linear_backward(grad(rows=0, accumulate=1), None, 0, None) == anvil.OK
    assert L.anvil_gated_linear_backward(grad(dx=0, dgate=0, dup=0), None, 0, None) == anvil.OK
    assert L.anvil_gated_linear_backward(grad(rows=0, dup=8 * G), None, 0, None) == anvil.ERR_ALIAS
    for f in (L.anvil_gated_linear_forward, L.anvil_gated_linear_backward):
        assert f(None, None, 0, None) == anvil.ERR_INVALID_ARG


def test_structures_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(anvil.HEADER).read(), flags=re.S)
    for cls, name in ((anvil.GatedDesc, "anvil_gated_desc"), (anvil.GatedGradDesc, "anvil_gated_grad_desc")):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
        fields = [f for decl in body.split(";") for f in re.findall(r"(\w+)\s*(?:,|$)", decl.strip())]
        assert fields == [f for f, _ in cls._fields_], name


def test_binding_refusals():
    import torch
    bf = torch.bfloat16
    x, w = torch.zeros((4, 8), dtype=bf), torch.zeros((6, 8), dtype=bf)
    z = torch.zeros((4, 6), dtype=bf)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.gated_linear_forward(x, w, w)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.gated_linear_backward(z, x, w, w, z, z)
    with pytest.raises(ValueError, match="requires grad"):
        anvil.gated_linear_forward(x, w.clone().requires_grad_(), w)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        anvil.gated_linear_forward(x.float(), w.float(), w.float())
    with pytest.raises(ValueError, match="x's type"):
        anvil.gated_linear_forward(x, w, w.half())
    with pytest.raises(ValueError, match=r"\[n, 8\]"):
        anvil.gated_linear_forward(x, w[:, :7], w)
    with pytest.raises(ValueError, match="gate's shape"):
        anvil.gated_linear_forward(x, w, w[:5])
    with pytest.raises(ValueError, match="all by rows or all by columns"):
        anvil.gated_linear_forward(x, w, torch.zeros((8, 6), dtype=bf).t())
    with pytest.raises(ValueError, match="activation must be"):
        anvil.gated_linear_forward(x, w, w, activation="swish")
    with pytest.raises(ValueError, match="preact_up must have"):
        anvil.gated_linear_backward(z, x, w, w, z, z[:3])
    with pytest.raises(ValueError, match="given together"):
        anvil.gated_linear_backward(z, x, w, w, z, z, dgate=w)
    with pytest.raises(ValueError, match="accumulate needs"):
        anvil.gated_linear_backward(z, x, w, w, z, z, accumulate=True)
    with pytest.raises(ValueError, match="both fp32"):
        anvil.gated_linear_backward(z, x, w, w, z, z, dgate=w, dup=w.float())
    with pytest.raises(ValueError, match="all by rows or all by columns"):
        anvil.gated_linear_backward(z, x, w, w, z, z, dgate=torch.zeros((8, 6), dtype=bf).t(), dup=w)
    with pytest.raises(ValueError, match="dz_parts"):
        anvil.gated_linear_backward(z, x, w, w, z, z, dz_parts=3)
