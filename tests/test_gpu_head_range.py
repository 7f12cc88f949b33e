"""GPU tests of the head's cross entropy at the ends of its range, against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, make_weight, randn  # noqa: E402,F401
from test_gpu_head import backward_check, make_targets  # noqa: E402


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_row_gradients_that_are_not_finite(A, bad):  # noqa: F811
    """fp16 holds the logits' gradients over the largest row gradient: of the finite ones, so that a row that is not
    does not take the others' digits."""
    rows, vocab, k = 90, 500, 64
    x, w = randn(1, rows, k, scale=2.0, dtype="f16"), make_weight(2, vocab, k, "f16", False)
    t, gl = make_targets(3, rows, vocab), randn(4, rows, scale=1e-4)
    _, lse = A.linear_cross_entropy(x, w, t)
    gl[11], t[11] = bad, 77
    dx, dw = A.linear_cross_entropy_backward(x, w, t, lse, gl)
    keep = torch.arange(rows, device="cuda") != 11
    assert not torch.isfinite(dx[11]).any() and not torch.isfinite(dw[77]).any()
    backward_check(x[keep], w, t[keep], lse[keep], gl[keep], "f16", "f16", (dx[keep], None))
