"""The gated layer's gradients of the last rows of a long batch, in fp32, against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, make_weight, randn  # noqa: E402,F401
from test_gpu_gated import backward_check  # noqa: E402


def test_fp32_gradients_past_32_bit_offsets(A):  # noqa: F811
    """Rows whose elements lie past 2^31: the rows alone give the same dx, and both calls' fp32 weight gradients
    are the definition's."""
    rows, n, k = (1 << 25) + 5, 72, 64
    x = torch.zeros(rows, k, device="cuda", dtype=torch.bfloat16)
    dy, g, u = (torch.zeros(rows, n, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    x[-300:] = randn(1, 300, k, dtype="bf16")
    for i, t in enumerate((dy, g, u)):
        t[-300:] = randn(4 + i, 300, n, dtype="bf16")
    wg, wu = make_weight(2, n, k, "bf16", False), make_weight(3, n, k, "bf16", False)
    got = A.gated_linear_backward(dy, x, wg, wu, g, u, dweight_dtype=torch.float32)
    tail = [t[-300:] for t in (dy, x)] + [wg, wu] + [t[-300:] for t in (g, u)]
    small = A.gated_linear_backward(*tail, dweight_dtype=torch.float32)
    backward_check(*tail, "silu", "bf16", "f32", small)
    backward_check(*tail, "silu", "bf16", "f32", (got[0][-300:], got[1], got[2]))
    assert not got[0][:-300].any() and torch.equal(got[0][-300:], small[0])
    assert A.device_error() == A.OK
