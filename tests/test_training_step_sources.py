"""What the kernels of a training step's operators rely on and a run cannot show, read from their sources,
and their refusals in grad mode (no GPU needed)."""
import re

import pytest

from test_block_sources import LOAD, code

NEW = ["anvil_linear.cuh", "anvil_gated.cu", "anvil_head.cu", "anvil_adamw.cu"]


@pytest.mark.parametrize("name", NEW)
def test_nothing_is_loaded_before_the_wait(name):
    """As in the other operators: what an earlier kernel may still write is loaded after the wait."""
    text = code(name)
    waits = [m.start() for m in re.finditer(r"^ *(?:if \(!p\.overlap_previous\) )?pdl_wait_previous\(\);", text, re.M)]
    assert waits
    for at in waits:
        start = text.rfind("\n__", 0, at)
        body = re.sub(r"\ba\.t\[[^]]*\]|full_bar\[\w+\]|empty_bar\[\w+\]|armed\[\w+\]", "", text[start:at])  # parameters, barriers
        assert not LOAD.search(body), body[-400:]


@pytest.mark.parametrize("name", NEW + ["anvil_multi.cu", "anvil_round.cuh"])
def test_loads_are_coherent(name):
    assert not re.search(r"__ldg\(|ld\.global\.nc", code(name))


def test_grad_mode():
    torch = pytest.importorskip("torch")
    anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")
    bf = torch.bfloat16
    x, w, z, t, f = torch.zeros(4, 8, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(4, 6, dtype=bf), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    calls = {
        "gated_linear_forward": (anvil.gated_linear_forward, (x, w, w.clone())),
        "gated_linear_backward": (anvil.gated_linear_backward, (z, x, w, w.clone(), z.clone(), z.clone())),
        "linear_cross_entropy": (anvil.linear_cross_entropy, (x, w, t)),
        "linear_cross_entropy_backward": (anvil.linear_cross_entropy_backward, (x, w, t, f, f.clone())),
    }
    for name, (call, tensors) in calls.items():
        for i, one in enumerate(tensors):
            if not one.is_floating_point():
                continue
            args = [u.clone().requires_grad_() if j == i else u for j, u in enumerate(tensors)]
            with pytest.raises(ValueError, match=name + ": a tensor requires grad"):
                call(*args)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # past the check
                call(*args)
