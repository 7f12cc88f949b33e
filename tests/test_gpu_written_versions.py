"""GPU tests that a graph which saved a tensor refuses it once a call has written to it: the tensors that the
training step's operators are given to write to."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, make_weight, randn  # noqa: E402,F401


def test_adamw(A):  # noqa: F811
    p, g = torch.zeros(600, device="cuda", dtype=torch.bfloat16), torch.ones(600, device="cuda")
    m, v, s = A.adamw_state(p, 8)
    low = torch.zeros(600, device="cuda", dtype=torch.int16)
    out = [torch.empty(600, device="cuda")], [torch.empty(600, device="cuda")]
    written, read = [p, m, v, s, low], [g]
    before = [t._version for t in written + read]
    A.adamw_step([p], [g], [m], [v], 1e-3, 1, mantissas=[low], scales=[s])
    after = [t._version for t in written + read]
    assert all(b > a for a, b in zip(before[:5], after)) and after[5] == before[5]
    before = [t._version for t in (m, v, s, out[0][0], out[1][0])]
    A.adamw_values([m], [v], [s], out=out)
    after = [t._version for t in (m, v, s, out[0][0], out[1][0])]
    assert after[:3] == before[:3] and after[3] > before[3] and after[4] > before[4]


def refused(tensor, call):
    """A graph that saved the tensor's values cannot go back after the call."""
    w = torch.ones(1, device="cuda", requires_grad=True)
    y = (w * tensor).sum()
    with torch.no_grad():
        call()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_results_given(A):  # noqa: F811
    bf = torch.bfloat16
    x, a, b = randn(1, 40, 64, dtype="bf16"), make_weight(2, 96, 64, "bf16", False), make_weight(3, 96, 64, "bf16", False)
    out, dy = torch.empty(40, 96, device="cuda", dtype=bf), randn(4, 40, 96, dtype="bf16")
    refused(out, lambda: A.gated_linear_forward(x, a, b, out=out))
    _, g, u = A.gated_linear_forward(x, a, b, save_preact=True)
    da, db = torch.zeros(96, 64, device="cuda"), torch.zeros(96, 64, device="cuda")
    for t in (da, db):
        refused(t, lambda: A.gated_linear_backward(dy, x, a, b, g, u, dgate=da, dup=db, accumulate=True))
    t, gl, dw = torch.zeros(40, device="cuda", dtype=torch.int64), torch.ones(40, device="cuda"), torch.zeros(96, 64, device="cuda")
    _, lse = A.linear_cross_entropy(x, a, t)
    refused(dw, lambda: A.linear_cross_entropy_backward(x, a, t, lse, gl, dweight=dw, accumulate=True))
    # what a call only reads stays good
    w = torch.ones(1, device="cuda", requires_grad=True)
    y = (w * x).sum() + (w * lse).sum()
    with torch.no_grad():
        A.linear_cross_entropy_backward(x, a, t, lse, gl)
    y.backward()
