"""GPU tests of the cross entropy's gradient where the vocabulary goes in several pieces, against 64 bits (bars
as in test_gpu_head.py).  How many pieces a call took is read from its launches."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_block_ops import A, DT, make_weight, randn  # noqa: E402,F401
from test_gpu_head import backward_check, make_targets  # noqa: E402

ROWS, VOCAB, K = 20000, 33001, 73  # 1.3 GB of logits' gradients in 16 bits: three pieces, the last one narrower and odd


def pieces_of(A, call):  # noqa: F811
    with A.profile() as prof:
        result = call()
        torch.cuda.synchronize()
    kinds = [k for k, _ in prof.records]
    return kinds.count("head_product"), result


def inputs(seed, dtype, transposed, pad=0, offset=0, rows=ROWS, vocab=VOCAB, k=K):
    x = randn(seed, rows, k, scale=2.0, dtype=dtype, pad=pad, offset=offset)
    return x, make_weight(seed + 1, vocab, k, dtype, transposed, pad, offset), make_targets(seed + 2, rows, vocab), randn(seed + 3, rows, scale=1.0 / rows)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_three_pieces(A, transposed, dtype):  # noqa: F811
    """Odd sizes, aligned and unaligned operands, 16-bit and fp32 weight gradients."""
    for seed, k, pad, off, dw_type in ((1, K, 0, 0, "f32"), (5, 72, 0, 0, dtype), (9, K, 1, 1, dtype), (13, 80, 8, 8, "f32")):
        x, w, t, gl = inputs(seed, dtype, transposed, pad, off, k=k)
        t[3], t[4] = 11007, 11008  # either side of a piece's end
        _, lse = A.linear_cross_entropy(x, w, t)
        n, got = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=DT[dw_type]))
        assert n == 3
        backward_check(x, w, t, lse, gl, dtype, dw_type, got)
        del got
    assert A.device_error() == A.OK


@pytest.mark.parametrize("transposed", [False, True])
def test_one_of_the_gradients(A, transposed):  # noqa: F811
    x, w, t, gl = inputs(21, "bf16", transposed)
    _, lse = A.linear_cross_entropy(x, w, t)
    n, got = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dweight=False))
    assert n == 3 and got[1] is None
    backward_check(x, w, t, lse, gl, "bf16", "bf16", got)
    n, got = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dx=False))
    assert n == 3 and got[0] is None
    backward_check(x, w, t, lse, gl, "bf16", "bf16", got)


@pytest.mark.parametrize("dw_type", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_accumulate(A, transposed, dw_type):  # noqa: F811
    """Added to what is there, in rows of a wider matrix; what is beside it stays."""
    x, w, t, gl = inputs(31, "bf16", transposed)
    _, lse = A.linear_cross_entropy(x, w, t)
    full = randn(35, *((K + 2, VOCAB + 19) if transposed else (VOCAB + 2, K + 19)), scale=0.1, dtype=dw_type)
    inner = full[1:-1, 8:-11]
    dw = inner.t() if transposed else inner
    base, before = dw.clone(), full.clone()
    n, got = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight=dw, accumulate=True))
    assert n == 3 and got[1].data_ptr() == dw.data_ptr()
    backward_check(x, w, t, lse, gl, "bf16", dw_type, got, base)
    inner.copy_(before[1:-1, 8:-11])
    assert torch.equal(full, before)


def test_the_same_bits_each_time(A):  # noqa: F811
    """d's buffer is taken again by the next piece while early launches are under way: calls one after the
    other, and replays of a graph, leave the same bits."""
    x, w, t, gl = inputs(41, "bf16", False)
    _, lse = A.linear_cross_entropy(x, w, t)
    call = lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl)  # noqa: E731
    want = call()
    for _ in range(4):
        got = call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_column_that_cannot_be(A):  # noqa: F811
    """Logits of -inf in the second piece: no gradient there, the others' as without that column."""
    x, w, t, gl = inputs(51, "bf16", False, k=64)
    x[:, 0] = 1.0
    w[20000, 0] = -float("inf")
    t[t == 20000] = 5
    _, lse = A.linear_cross_entropy(x, w, t)
    n, got = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, need_dx=False, dweight_dtype=torch.float32))
    assert n == 3 and not got[1][20000].any()
    keep = torch.arange(VOCAB, device="cuda") != 20000
    backward_check(x, w[keep], t - (t > 20000).long(), lse, gl, "bf16", "f32", (None, got[1][keep]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_pieces_of_long_contractions(A, transposed, dtype):  # noqa: F811
    """More than 1024 features, where the logits are added up from several chains.  A hundred rows count, so that the
    definition needs no others."""
    k = 1100
    x, w, t, gl = inputs(61, dtype, transposed, k=k)
    keep = torch.zeros(ROWS, dtype=torch.bool, device="cuda")
    keep[torch.arange(100, device="cuda") * 199 + 7] = True
    t[~keep] = -1
    t[keep] = torch.arange(100, device="cuda") * 330 + 5
    _, lse = A.linear_cross_entropy(x, w, t)
    n, (dx, dw) = pieces_of(A, lambda: A.linear_cross_entropy_backward(x, w, t, lse, gl, dweight_dtype=torch.float32))
    assert n == 3 and not dx[~keep].any()
    backward_check(x[keep], w, t[keep], lse[keep], gl[keep], dtype, "f32", (dx[keep], dw))
