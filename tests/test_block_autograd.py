"""The operators around the banks leave nothing for autograd, so they refuse a tensor that asks for
a gradient where grad mode is on, before anything else of the call (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
anvil = pytest.importorskip("polynomial_matrix_whitening_gb300.anvil", reason="libanvil.so not built")

BF = torch.bfloat16


def calls():
    """name -> (call, its tensors)"""
    x, w, dy, r = torch.zeros(4, 8), torch.zeros(6, 8, dtype=BF), torch.zeros(4, 6, dtype=BF), torch.zeros(4)
    v, b, t = torch.zeros(8), torch.zeros(6), torch.zeros(4, dtype=torch.int64)
    xb = x.to(BF)
    return {
        "layernorm_forward": (lambda x, w, b: anvil.layernorm_forward(x, w, b), (x, v, v.clone())),
        "layernorm_backward": (lambda dy, x, m, s, w, res: anvil.layernorm_backward(dy, x, m, s, w, residual_grad=res),
                               (x, x.clone(), r, r.clone(), v, x.clone())),
        "linear_forward": (lambda x, w, b, res: anvil.linear_forward(x, w, b, residual=res), (xb, w, b, dy)),
        "linear_backward": (lambda dy, x, w, z, dw, db: anvil.linear_backward(dy, x, w, preact=z, activation="silu", dweight=dw,
                                                                              dbias=db),
                            (dy, xb, w, dy.clone(), w.clone(), b)),
        "token_logprobs": (lambda x, t: anvil.token_logprobs(x, t), (x, t)),
        "token_logprobs_backward": (lambda x, t, lse, gl, e, gh: anvil.token_logprobs_backward(x, t, lse, gl, entropy=e,
                                                                                               grad_entropy=gh),
                                    (x, t, r, r.clone(), r.clone(), r.clone())),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_grad_mode(name):
    call, tensors = calls()[name]
    for i, t in enumerate(tensors):
        if not t.is_floating_point():
            continue
        args = [u.clone().requires_grad_() if j == i else u for j, u in enumerate(tensors)]
        with pytest.raises(ValueError, match=name + ": a tensor requires grad"):
            call(*args)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # past the check
            call(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        call(*tensors)


class Linear(torch.autograd.Function):
    """The linear layer inside an autograd graph, with its own backward call."""

    @staticmethod
    def forward(ctx, x, w, b):
        y, z = anvil.linear_forward(x, w, b, activation="silu", save_preact=True)
        ctx.save_for_backward(x, w, z)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        return anvil.linear_backward(dy.contiguous(), x, w, preact=z, activation="silu")


@pytest.mark.gpu
def test_inside_an_autograd_function():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(s, generator=gen, device="cuda").to(BF).requires_grad_() for s in ((300, 64), (96, 64)))
    b = torch.randn(96, generator=gen, device="cuda").requires_grad_()
    y = Linear.apply(x, w, b)
    dy = torch.randn(300, 96, generator=gen, device="cuda").to(BF)
    y.backward(dy)
    with torch.no_grad():
        want, z = anvil.linear_forward(x, w, b, activation="silu", save_preact=True)
        dx, dw, db = anvil.linear_backward(dy, x, w, preact=z, activation="silu")
    assert torch.equal(y, want) and torch.equal(x.grad, dx) and torch.equal(w.grad, dw) and torch.equal(b.grad, db)
    with pytest.raises(ValueError, match="requires grad"):
        anvil.linear_forward(x, w, b)
