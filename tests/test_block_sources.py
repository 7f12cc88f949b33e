"""What the operators' kernels rely on and a run cannot show, read from their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "polynomial_matrix_whitening_gb300", "csrc")
LOAD = re.compile(r"Elem<\w+>::load\(|__ld\w+\(|\bldg_stream\(|\)\[\w+\]|\b(?:mean|rstd|part|lse|entropy|targets|bias)\[")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["anvil_linear.cu", "anvil_norm.cu", "anvil_logprob.cu"])
def test_nothing_is_loaded_before_the_wait(name):
    """A kernel may start before the one ahead of it has ended: what it loads, an earlier kernel may
    still be writing, until it has waited."""
    text = code(name)
    waits = [m.start() for m in re.finditer(r"^ *(?:if \(!p\.overlap_previous\) )?pdl_wait_previous\(\);", text, re.M)]
    assert waits
    for at in waits:
        start = text.rfind("\n__", 0, at)  # the function's own line
        assert not LOAD.search(text[start:at]), text[start:at][-400:]


@pytest.mark.parametrize("name", ["anvil_linear.cu", "anvil_norm.cu", "anvil_logprob.cu", "anvil_types.cuh",
                                  "anvil_elementwise.cu", "anvil_tail.cu", "anvil_adam.cu", "anvil_gemm.cu"])
def test_loads_are_coherent(name):
    """The non-coherent path is for data that no one writes while the kernel runs; a kernel launched
    early runs beside the one that writes its inputs."""
    assert not re.search(r"__ldg\(|ld\.global\.nc", code(name))
