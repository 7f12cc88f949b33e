"""GPU test of the example: the operators and the bank step together, as a training program
runs them (polynomial_matrix_whitening_gb300/train_example.py)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from polynomial_matrix_whitening_gb300 import train_example

    return train_example


def reference(model, tokens, targets):
    """Loss, entropy and gradients of the same model in 64 bits."""
    leaf = lambda t: t.detach().double().requires_grad_()  # noqa: E731
    bank, head = leaf(model.bank), leaf(model.head.value)
    gains, shifts = [leaf(g.value) for g in model.gains], [leaf(s.value) for s in model.shifts]
    norm = lambda x, i: torch.nn.functional.layer_norm(x, x.shape[-1:], gains[i], shifts[i], 1e-5)  # noqa: E731
    x = model.embedding[tokens].double()
    for i in range(model.blocks):
        x = x + norm(x, i).matmul(bank[2 * i].t()).clamp_min(0).square().matmul(bank[2 * i + 1])
    logp = torch.log_softmax(norm(x, -1).matmul(head.t()), 1)
    loss = -logp.gather(1, targets[:, None]).mean()
    loss.backward()
    entropy = -(logp.exp() * logp).sum(1).mean()
    return loss.detach(), entropy.detach(), bank.grad, head.grad, [(g.grad, s.grad) for g, s in zip(gains, shifts)]


def test_example_gradients(E):
    model, data = E.Model(vocab=503, dim=256, hidden=512, blocks=2, seed=3), E.Data(503)
    tokens, targets = data.batch(701)
    (loss, entropy), (dhead, norms) = model.loss_and_gradients(tokens, targets)
    rloss, rentropy, rbank, rhead, rnorms = reference(model, tokens, targets)
    # A path from a weight to the loss and back passes at most twelve tensors that are rounded
    # to bf16, 2^-9 of a value each (2^-8 where it is squared next).
    bound = 12 * 2.0 ** -8

    def close(got, ref, what):
        assert float((got.double() - ref).norm()) <= bound * float(ref.norm()), what

    # the logits of one row, at most 6 in magnitude, carry the roundings of their path
    assert abs(float(loss) - float(rloss)) < 6 * bound and abs(float(entropy) - float(rentropy)) < 6 * bound
    for i in range(4):
        close(model.grad[i], rbank[i], f"bank {i}")
    close(dhead, rhead, "head")
    for i, (got, ref) in enumerate(zip(norms, rnorms)):
        close(got[0], ref[0], f"gain {i}")
        close(got[1], ref[1], f"shift {i}")


def test_example_learns(E):
    """The loss falls from above log(vocab) to below half of it, and generation follows the map."""
    model, data = E.Model(vocab=503, dim=256, hidden=512, blocks=2), E.Data(503)
    losses = E.train(model, data, 40, 2000)
    assert losses[0] > 6.0 and losses[-1] < 3.0
    got = model.generate(17, 6)
    follow = data.follow.tolist()
    usual = sum(t == follow[p] for p, (t, _) in zip([17] + [t for t, _ in got], got))
    assert usual >= 4
    for token, best in got:
        assert best[0][0] == token and all(a[1] >= b[1] for a, b in zip(best, best[1:]))


def test_example_step_in_a_graph(E):
    """Forward and backward of a step captured once give the same bits when replayed."""
    model, data = E.Model(vocab=503, dim=256, hidden=512, blocks=2, seed=5), E.Data(503)
    tokens, targets = data.batch(300)
    want, (dhead, _) = model.loss_and_gradients(tokens, targets)
    bank = model.grad.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, (dhead2, _) = model.loss_and_gradients(tokens, targets)
    model.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(model.grad, bank) and torch.equal(dhead2, dhead)
    assert float(got[0]) == float(want[0]) and float(got[1]) == float(want[1])
