"""GPU tests of the operators of a training step together, as the example's options run them: gated blocks,
the head's cross entropy without logits, AdamW over the head and the norms at once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OPTIONS = [dict(gated=True), dict(fused_loss=True), dict(gated=True, fused_loss=True, adamw=8), dict(adamw=32)]
NAMES = ["-".join(o) for o in OPTIONS]


@pytest.fixture(scope="module")
def E():
    from polynomial_matrix_whitening_gb300 import train_example

    return train_example


def reference(model, tokens, targets):
    """Loss and gradients of the same model in 64 bits."""
    leaf = lambda t: t.detach().double().requires_grad_()  # noqa: E731
    bank, head = leaf(model.bank), leaf(model.head.value)
    gains, shifts = [leaf(g.value) for g in model.gains], [leaf(s.value) for s in model.shifts]
    norm = lambda x, i: torch.nn.functional.layer_norm(x, x.shape[-1:], gains[i], shifts[i], 1e-5)  # noqa: E731
    x = model.embedding[tokens].double()
    for i in range(model.blocks):
        h = norm(x, i)
        if model.gated:
            a = torch.nn.functional.silu(h @ bank[3 * i].t()) * (h @ bank[3 * i + 1].t())
            x = x + a @ bank[3 * i + 2]
        else:
            x = x + (h @ bank[2 * i].t()).clamp_min(0).square() @ bank[2 * i + 1]
    loss = torch.nn.functional.cross_entropy(norm(x, -1) @ head.t(), targets)
    loss.backward()
    return loss.detach(), bank.grad, head.grad, [(g.grad, s.grad) for g, s in zip(gains, shifts)]


@pytest.mark.parametrize("options", OPTIONS, ids=NAMES)
def test_gradients(E, options):
    model, data = E.Model(vocab=503, dim=256, hidden=512, blocks=2, seed=3, **options), E.Data(503)
    tokens, targets = data.batch(701)
    (loss, entropy), (dhead, norms) = model.loss_and_gradients(tokens, targets)
    assert (entropy is None) == bool(options.get("fused_loss"))
    rloss, rbank, rhead, rnorms = reference(model, tokens, targets)
    # A path from a weight to the loss and back passes at most fourteen tensors that are rounded to
    # bf16, 2^-9 of a value each (2^-8 where it is squared or multiplied by another one next).
    bound = 14 * 2.0 ** -8

    def close(got, ref, what):
        assert float((got.double() - ref).norm()) <= bound * float(ref.norm()), what

    assert abs(float(loss) - float(rloss)) < 6 * bound  # (logits of at most 6 carry the roundings of their path)
    for i in range(len(rbank)):
        close(model.grad[i], rbank[i], f"bank {i}")
    close(dhead, rhead, "head")
    for i, (got, ref) in enumerate(zip(norms, rnorms)):
        close(got[0], ref[0], f"gain {i}")
        close(got[1], ref[1], f"shift {i}")


def test_fused_loss_is_the_loss(E):
    """The same hidden values and head through logits and without them: the loss to fp32 accuracy of bf16
    logits (2^-9 of each, at most 6), the gradients to the roundings of dlogits (2^-9 either way)."""
    tokens, targets = E.Data(5003).batch(900)
    plain, fused = (E.Model(vocab=5003, dim=256, hidden=512, blocks=1, seed=4, fused_loss=f) for f in (False, True))
    (a, _), (da, _) = plain.loss_and_gradients(tokens, targets)
    (b, _), (db, _) = fused.loss_and_gradients(tokens, targets)
    assert abs(float(a) - float(b)) < 6 * 2.0 ** -8
    assert float((da - db).norm()) <= 4 * 2.0 ** -8 * float(da.norm())
    assert float((plain.grad - fused.grad).norm()) <= 8 * 2.0 ** -8 * float(plain.grad.norm())


@pytest.mark.parametrize("bits", [8, 32])
def test_step_of_head_and_norms(E, bits):
    """One step from zero moments moves every value by lr times its gradient's sign, where the
    gradient counts beside eps; with 8 bits as with 32 (a step takes the unrounded moments)."""
    model, data = E.Model(vocab=503, dim=256, hidden=512, blocks=2, seed=5, gated=True, fused_loss=True, adamw=bits), E.Data(503)
    tokens, targets = data.batch(2000)
    _, (dhead, norms) = model.loss_and_gradients(tokens, targets)
    master = lambda p: (p.value.view(torch.int16).int() << 16 | p.mantissa.int() & 0xFFFF).view(torch.float32)  # noqa: E731
    before, gain = master(model.head).clone(), model.gains[0].value.clone()
    model.step(tokens, targets, lr=2e-3)
    for now, old, g in ((master(model.head), before, dhead), (model.gains[0].value, gain, norms[0][0])):
        # m = 0.1 g and sqrt(v) = sqrt(0.05) |g| with their corrections: g / (|g| + eps), fp32 roundings of
        # the value (2^-24) and of the step (2^-20 of it covers a dozen)
        want = old.double() - 2e-3 * g.double() / (g.double().abs() + 1e-8)
        assert ((now.double() - want).abs() <= 2.0 ** -23 * old.double().abs() + 2e-3 * 2.0 ** -20).all()


@pytest.mark.parametrize("options", OPTIONS, ids=NAMES)
def test_runs(E, options, capsys):
    """Several steps and generation, through the command line."""
    argv = ["--steps", "3", "--tokens", "300", "--vocab", "503", "--dim", "256", "--hidden", "512", "--blocks", "1"]
    argv += (["--gated"] if "gated" in options else []) + (["--fused-loss"] if "fused_loss" in options else [])
    argv += ["--adamw", str(options["adamw"])] if "adamw" in options else []
    E.main(argv)
    out = capsys.readouterr().out
    assert out.count("step") == 2 and out.count("->") == 4 and "nan" not in out
    assert ("entropy" in out) == ("fused_loss" not in options)


def test_step_in_a_graph(E):
    """Forward, backward and the AdamW step captured once: replayed, the same bits as run."""
    from polynomial_matrix_whitening_gb300 import anvil
    models = [E.Model(vocab=503, dim=256, hidden=512, blocks=2, seed=6, gated=True, fused_loss=True, adamw=8) for _ in range(2)]
    tokens, targets = E.Data(503).batch(300)

    def step(model, scalars=None):
        _, (dhead, norms) = model.loss_and_gradients(tokens, targets)
        ps = [model.head] + model.gains + model.shifts
        ms, vs, scales = zip(*(p.state for p in ps))
        grads = [dhead] + [g for g, _ in norms] + [g for _, g in norms]
        anvil.adamw_step([p.value for p in ps], grads, ms, vs, 2e-3, 1, mantissas=[p.mantissa for p in ps], scales=scales,
                         scalars=scalars)

    run, replayed = models
    scalars = torch.tensor(anvil.adamw_scalars(2e-3, 1), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(replayed, scalars)
    for t in (1, 2, 3):
        scalars.copy_(torch.tensor(anvil.adamw_scalars(2e-3 / t, t)))
        graph.replay()
        step(run, scalars)
    torch.cuda.synchronize()
    for a, b in zip([run.head] + run.gains, [replayed.head] + replayed.gains):
        assert torch.equal(a.value, b.value)
        for s, t in zip(a.state, b.state):
            assert s is None or np.array_equal(s.view(torch.uint8).cpu().numpy(), t.view(torch.uint8).cpu().numpy())
    assert torch.equal(run.head.mantissa, replayed.head.mantissa) and torch.equal(run.grad, replayed.grad)
