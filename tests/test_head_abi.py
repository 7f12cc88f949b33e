"""The head's cross entropy, what needs no GPU: refusals before any CUDA call (the pointers are fake),
workspace sizes, the binding's refusals."""
import re

import pytest

anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")
L = anvil.library()
G = 1 << 40  # fake, aligned device addresses far apart


def fill(cls, base, kw):
    base.update(kw)
    return cls(*[base[k] for k, _ in cls._fields_])


def desc(**kw):
    return fill(anvil.HeadDesc, dict(x=G, weight=2 * G, targets=3 * G, loss=4 * G, lse=5 * G, rows=100, ldx=64, ldw=64, vocab=1000,
                                     k=64, dtype=1, targets_int64=1, weight_transposed=0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), anvil.ERR_INVALID_ARG), (dict(weight=0), anvil.ERR_INVALID_ARG), (dict(targets=0), anvil.ERR_INVALID_ARG),
    (dict(dtype=0), anvil.ERR_INVALID_ARG), (dict(vocab=0), anvil.ERR_INVALID_ARG), (dict(k=0), anvil.ERR_INVALID_ARG),
    (dict(rows=-1), anvil.ERR_INVALID_ARG), (dict(ldx=63), anvil.ERR_INVALID_ARG), (dict(ldw=63), anvil.ERR_INVALID_ARG),
    (dict(weight_transposed=1), anvil.ERR_INVALID_ARG), (dict(vocab=(1 << 24) + 1), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(rows=1 << 30, vocab=1 << 24), anvil.ERR_UNSUPPORTED_SHAPE), (dict(k=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(x=G + 1), anvil.ERR_ALIGNMENT), (dict(targets=3 * G + 4), anvil.ERR_ALIGNMENT), (dict(loss=4 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(loss=G), anvil.ERR_ALIAS), (dict(lse=4 * G + 4), anvil.ERR_ALIAS), (dict(lse=3 * G + 8), anvil.ERR_ALIAS),
    (dict(lse=2 * G + 64), anvil.ERR_ALIAS), (dict(ws=0), anvil.ERR_WORKSPACE), (dict(wsb=1000), anvil.ERR_WORKSPACE),
    (dict(ws=(1 << 50) + 8), anvil.ERR_ALIGNMENT), (dict(ws=5 * G), anvil.ERR_ALIAS),
])
def test_forward_refusals(kw, code):
    ws, wsb = kw.pop("ws", 1 << 50), kw.pop("wsb", 1 << 40)
    assert L.anvil_linear_cross_entropy(desc(**kw), ws, wsb, None) == code


def grad(**kw):
    return fill(anvil.HeadGradDesc, dict(x=G, weight=2 * G, targets=3 * G, lse=4 * G, grad_loss=5 * G, dx=6 * G, dweight=7 * G,
                                         rows=100, ldx=64, ldw=64, lddx=64, lddw=64, vocab=1000, k=64, dtype=1, targets_int64=1,
                                         dweight_dtype=1, weight_transposed=0, accumulate=0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), anvil.ERR_INVALID_ARG), (dict(weight=0), anvil.ERR_INVALID_ARG), (dict(targets=0), anvil.ERR_INVALID_ARG),
    (dict(lse=0), anvil.ERR_INVALID_ARG), (dict(grad_loss=0), anvil.ERR_INVALID_ARG), (dict(dtype=0), anvil.ERR_INVALID_ARG),
    (dict(dweight_dtype=2), anvil.ERR_INVALID_ARG), (dict(lddx=63), anvil.ERR_INVALID_ARG), (dict(lddw=63), anvil.ERR_INVALID_ARG),
    (dict(ldx=63), anvil.ERR_INVALID_ARG), (dict(dweight=7 * G + 1), anvil.ERR_ALIGNMENT), (dict(lse=4 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(dx=G), anvil.ERR_ALIAS), (dict(dweight=2 * G), anvil.ERR_ALIAS), (dict(dx=4 * G), anvil.ERR_ALIAS),
    (dict(dweight=6 * G + 128), anvil.ERR_ALIAS), (dict(ws=0), anvil.ERR_WORKSPACE), (dict(wsb=64), anvil.ERR_WORKSPACE),
    (dict(ws=(1 << 50) + 64), anvil.ERR_ALIGNMENT), (dict(ws=7 * G), anvil.ERR_ALIAS),
])
def test_backward_refusals(kw, code):
    ws, wsb = kw.pop("ws", 1 << 50), kw.pop("wsb", 1 << 40)
    assert L.anvil_linear_cross_entropy_backward(grad(**kw), ws, wsb, None) == code


def test_workspaces_and_no_work():
    need = lambda **kw: L.anvil_linear_cross_entropy_workspace_bytes(desc(**kw))  # noqa: E731
    assert need(rows=1000) >= 8 * 1000 * 16 and need(rows=0) == 0 and need(loss=0, lse=0) == 0
    assert need(weight=2 * G + 2) == need() + 1000 * 64 * 2
    back = lambda **kw: L.anvil_linear_cross_entropy_backward_workspace_bytes(grad(**kw))  # noqa: E731
    assert back() >= 100 * 1000 * 2 and back(dx=0, dweight=0) == 0
    # the gradient of the logits is bounded: not 65536 rows of 1,000,000
    assert back(rows=1 << 16, vocab=1000000) < 2 << 30
    assert L.anvil_linear_cross_entropy(desc(rows=0), None, 0, None) == anvil.OK
    assert L.anvil_linear_cross_entropy(desc(loss=0, lse=0, targets=0), None, 0, None) == anvil.OK
    assert L.anvil_linear_cross_entropy_backward(grad(rows=0, accumulate=1), None, 0, None) == anvil.OK
    for f in (L.anvil_linear_cross_entropy, L.anvil_linear_cross_entropy_backward):
        assert f(None, None, 0, None) == anvil.ERR_INVALID_ARG


def test_structures_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(anvil.HEADER).read(), flags=re.S)
    for cls, name in ((anvil.HeadDesc, "anvil_head_desc"), (anvil.HeadGradDesc, "anvil_head_grad_desc")):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
        fields = [f for decl in body.split(";") for f in re.findall(r"(\w+)\s*(?:,|$)", decl.strip())]
        assert fields == [f for f, _ in cls._fields_], name


def test_kernel_kinds_match_the_header():
    text = open(anvil.HEADER).read()
    body = re.search(r"typedef enum \{([^{}]*)\} anvil_kernel_kind;", text).group(1)
    names = re.findall(r"ANVIL_KERNEL_(\w+) = (\d+)", body)
    assert [(n.lower(), int(i)) for n, i in names] == [(n, i) for i, n in enumerate(anvil.KERNEL_KINDS)]


def test_binding_refusals():
    import torch
    bf = torch.bfloat16
    x, w, t = torch.zeros((4, 8), dtype=bf), torch.zeros((60, 8), dtype=bf), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.linear_cross_entropy_backward(x, w, t, f, f)
    with pytest.raises(ValueError, match="requires grad"):
        anvil.linear_cross_entropy(x, w.clone().requires_grad_(), t)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        anvil.linear_cross_entropy(x.float(), w.float(), t)
    with pytest.raises(ValueError, match=r"\[vocab, 8\]"):
        anvil.linear_cross_entropy(x, torch.zeros((60, 9), dtype=bf), t)
    with pytest.raises(ValueError, match="targets must be"):
        anvil.linear_cross_entropy(x, w, t[:3])
    with pytest.raises(ValueError, match="targets must be"):
        anvil.linear_cross_entropy(x, w, f)
    with pytest.raises(ValueError, match="lse must be"):
        anvil.linear_cross_entropy_backward(x, w, t, f[:3], f)
    with pytest.raises(ValueError, match="grad_loss must be"):
        anvil.linear_cross_entropy_backward(x, w, t, f, f.double())
    with pytest.raises(ValueError, match="accumulate needs"):
        anvil.linear_cross_entropy_backward(x, w, t, f, f, accumulate=True)
    with pytest.raises(ValueError, match="dweight must be fp32"):
        anvil.linear_cross_entropy_backward(x, w, t, f, f, dweight_dtype=torch.float16)
