"""AdamW over many tensors, what needs no GPU: refusals before any CUDA call (the pointers are fake),
the scalars of a step, the binding's refusals."""
import ctypes
import math
import re

import pytest

anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")
L = anvil.library()
G = 1 << 36  # fake, aligned device addresses far apart


def tensor(**kw):
    base = dict(param=G, mantissa=0, grad=2 * G, exp_avg=3 * G, exp_avg_sq=4 * G, scales=0, count=1000, param_dtype=0, grad_dtype=0)
    base.update(kw)
    return anvil.AdamwTensor(*[base[k] for k, _ in anvil.AdamwTensor._fields_])


def step(tensors, d_scalars=None, n=None, **kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=1)
    base.update(kw)
    c = anvil.AdamwConfig(*[base[k] for k, _ in anvil.AdamwConfig._fields_])
    arr = (anvil.AdamwTensor * max(1, len(tensors)))(*tensors)
    return L.anvil_adamw_step(arr, len(tensors) if n is None else n, ctypes.byref(c), d_scalars, None)


@pytest.mark.parametrize("kw,code", [
    (dict(param=0), anvil.ERR_INVALID_ARG), (dict(grad=0), anvil.ERR_INVALID_ARG), (dict(exp_avg=0), anvil.ERR_INVALID_ARG),
    (dict(exp_avg_sq=0), anvil.ERR_INVALID_ARG), (dict(count=-1), anvil.ERR_INVALID_ARG),
    (dict(param_dtype=3), anvil.ERR_INVALID_ARG), (dict(grad_dtype=-1), anvil.ERR_INVALID_ARG),
    (dict(param_dtype=1, grad_dtype=2), anvil.ERR_INVALID_ARG), (dict(param_dtype=2, grad_dtype=1), anvil.ERR_INVALID_ARG),
    (dict(mantissa=5 * G), anvil.ERR_INVALID_ARG), (dict(mantissa=5 * G, param_dtype=2), anvil.ERR_INVALID_ARG),
    (dict(count=(1 << 40) + 1), anvil.ERR_UNSUPPORTED_SHAPE),
    (dict(param=G + 2), anvil.ERR_ALIGNMENT), (dict(param=G + 1, param_dtype=1), anvil.ERR_ALIGNMENT),
    (dict(grad=2 * G + 2), anvil.ERR_ALIGNMENT), (dict(exp_avg=3 * G + 2), anvil.ERR_ALIGNMENT),
    (dict(scales=5 * G + 2), anvil.ERR_ALIGNMENT), (dict(mantissa=5 * G + 1, param_dtype=1), anvil.ERR_ALIGNMENT),
    (dict(grad=G), anvil.ERR_ALIAS), (dict(exp_avg=G + 3996), anvil.ERR_ALIAS), (dict(exp_avg_sq=3 * G + 4), anvil.ERR_ALIAS),
    (dict(scales=3 * G + 996), anvil.ERR_ALIAS), (dict(mantissa=2 * G, param_dtype=1), anvil.ERR_ALIAS),
])
def test_tensor_refusals(kw, code):
    assert step([tensor(**kw)]) == code
    far = dict(param=11 * G, grad=12 * G, exp_avg=13 * G, exp_avg_sq=14 * G)
    assert step([tensor(**far), tensor(**kw)]) == code


def test_refusals_between_tensors():
    a = tensor()
    others = dict(param=11 * G, grad=12 * G, exp_avg=13 * G, exp_avg_sq=14 * G)
    for field, to in (("param", G + 3996), ("exp_avg", 2 * G), ("grad", G + 40), ("exp_avg_sq", 3 * G + 3996), ("scales", 4 * G)):
        assert step([a, tensor(**dict(others, **{field: to}))]) == anvil.ERR_ALIAS, field
        assert step([tensor(**dict(others, **{field: to})), a]) == anvil.ERR_ALIAS, field
    assert step([a, a]) == anvil.ERR_ALIAS  # the same tensor twice
    assert step([a], d_scalars=3 * G + 8) == anvil.ERR_ALIAS
    assert step([a], d_scalars=9 * G + 2) == anvil.ERR_ALIGNMENT


@pytest.mark.parametrize("kw", [dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=math.nan), dict(eps=-1e-8), dict(eps=math.nan),
                                dict(lr=math.inf), dict(weight_decay=math.nan), dict(grad_scale=math.inf), dict(step=0)])
def test_config_refusals(kw):
    assert step([tensor()], **kw) == anvil.ERR_INVALID_ARG
    assert step([], **kw) == anvil.ERR_INVALID_ARG


def test_counts_of_tensors():
    assert step([]) == anvil.OK and step([tensor(count=0, param=0, grad=0, exp_avg=0, exp_avg_sq=0)]) == anvil.OK
    assert step([tensor()], n=-1) == anvil.ERR_INVALID_ARG
    assert step([tensor()], n=(1 << 20) + 1) == anvil.ERR_UNSUPPORTED_SHAPE
    assert L.anvil_adamw_step(None, 1, ctypes.byref(anvil.AdamwConfig(1e-3, 0.9, 0.95, 1e-8, 0, 1, 1)), None, None) \
        == anvil.ERR_INVALID_ARG
    assert L.anvil_adamw_step(None, 0, None, None, None) == anvil.ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(exp_avg=0), anvil.ERR_INVALID_ARG), (dict(exp_avg_sq=0), anvil.ERR_INVALID_ARG), (dict(scales=0), anvil.ERR_INVALID_ARG),
    (dict(m=0), anvil.ERR_INVALID_ARG), (dict(v=0), anvil.ERR_INVALID_ARG), (dict(count=-1), anvil.ERR_INVALID_ARG),
    (dict(m=4 * G + 2), anvil.ERR_ALIGNMENT), (dict(scales=3 * G + 1), anvil.ERR_ALIGNMENT),
    (dict(m=G), anvil.ERR_ALIAS), (dict(v=4 * G), anvil.ERR_ALIAS), (dict(v=3 * G + 28), anvil.ERR_ALIAS),
    (dict(count=0, m=0, v=0), anvil.OK),
])
def test_values_refusals(kw, code):
    base = dict(exp_avg=G, exp_avg_sq=2 * G, scales=3 * G, m=4 * G, v=5 * G, count=1000)
    base.update(kw)
    s = anvil.AdamwState(*[base[k] for k, _ in anvil.AdamwState._fields_])
    assert L.anvil_adamw_values(ctypes.byref(s), 1, None) == code


def test_scalars():
    got = anvil.adamw_scalars(3e-4, 5, 0.9, 0.999, 0.1, 2.0)
    want = [3e-4 / (1 - 0.9 ** 5), (1 - 0.999 ** 5) ** -0.5, 1 - 3e-5, 2.0]
    assert all(abs(g - w) <= 2.0 ** -24 * w * (1 + 1e-6) for g, w in zip(got, want))
    with pytest.raises(anvil.AnvilError):
        anvil.adamw_scalars(3e-4, 0)


def test_structures_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(anvil.HEADER).read(), flags=re.S)
    for cls, name in ((anvil.AdamwTensor, "anvil_adamw_tensor"), (anvil.AdamwConfig, "anvil_adamw_config"),
                      (anvil.AdamwState, "anvil_adamw_state")):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
        fields = [f for decl in body.split(";") for f in re.findall(r"(\w+)\s*(?:,|$)", decl.strip())]
        assert fields == [f for f, _ in cls._fields_], name
    assert int(re.search(r"define ANVIL_ADAMW_BLOCK (\d+)", text).group(1)) == anvil.ADAMW_BLOCK


def test_binding_refusals():
    import torch
    p = torch.zeros(300)
    m, v, s = anvil.adamw_state(p, 8)
    assert m.dtype == torch.float8_e4m3fn and v.dtype == torch.uint8 and tuple(s.shape) == (2, 2)
    assert anvil.adamw_state(p)[2] is None
    with pytest.raises(ValueError, match="bits must be"):
        anvil.adamw_state(p, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.adamw_step([p], [p], [p], [p], 1e-3, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        anvil.adamw_values([m], [v], [s])
    with pytest.raises(ValueError, match="list of tensors"):
        anvil.adamw_step(p, [p], [p], [p], 1e-3, 1)
    with pytest.raises(ValueError, match="one tensor for each"):
        anvil.adamw_step([p], [p, p], [p], [p], 1e-3, 1)
    with pytest.raises(TypeError):
        anvil.adamw_step([p], [p], [p], [p], 1e-3, "first")
    anvil.adamw_step([], [], [], [], 1e-3, 1)
    assert anvil.adamw_values([], [], []) == ([], [])


def test_refusals_among_many_tensors():
    """Tensors in any order of addresses, arrays of all roles between each other: one overlap among them is found."""
    import random
    rng = random.Random(5)
    slots = list(range(1, 4 * 40 + 1))
    rng.shuffle(slots)

    def tensors(**kw):
        it = iter(slots)
        at = [[next(it) << 20 for _ in range(4)] for _ in range(40)]
        made = [tensor(param=a, grad=b, exp_avg=c, exp_avg_sq=d, count=1000) for a, b, c, d in at]
        for k, v in kw.items():
            setattr(made[17], k, v)
        return made
    for other in (3, 16, 18, 39):
        for field in ("param", "grad", "exp_avg", "exp_avg_sq"):
            lo = getattr(tensors()[other], field)
            assert step(tensors(param=lo + 3996)) == anvil.ERR_ALIAS
            assert step(tensors(exp_avg=lo - 3996)) == anvil.ERR_ALIAS
            if field != "grad":
                assert step(tensors(grad=lo + 8)) == anvil.ERR_ALIAS
