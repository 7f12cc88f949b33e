"""A small language model trained with libanvil, end to end on one GPU.

The operators around the banks as a training program uses them, next to the bank step:

    forward    x_0 = embedding;  per block  x += W_down act(W_up norm(x));  logits = W_head norm(x)
    loss       the mean of -log p(next token), entropy alongside
    backward   token log probabilities -> head -> norm -> blocks, the residual's gradient added
               inside the norm's backward pass, the weight gradients written as fp32 straight
               into the bank's gradient
    update     all W_up and W_down are one bank [2 * blocks, hidden, dim]: bank step and update
               tail; the head and the norms take the Adam step
    serving    one token at a time, with the likeliest alternatives

The data is synthetic: the next token follows from the current one by a fixed random map
nine times in ten, and is any token else.  The embedding is fixed.

    python -m polynomial_matrix_whitening_gb300.train_example [--steps N] [--tokens N] ...
"""
from __future__ import annotations

import argparse

import torch

from . import anvil

BF16, F32 = torch.bfloat16, torch.float32


class Adam:
    """An fp32 parameter with its moments; `value` is what the model computes with."""

    def __init__(self, init, compute=F32):
        self.master = init.to(F32).contiguous()
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.value = self.master if compute == F32 else self.master.to(compute)
        self.step = 0

    def update(self, grad, lr, beta1=0.9, beta2=0.95, eps=1e-8):
        self.step += 1
        scale = lr * (1 - beta2 ** self.step) ** 0.5 / (1 - beta1 ** self.step)
        anvil.adam_step(self.master, grad, self.m, self.v, beta1, beta2, eps, scale, 0.0)
        if self.value is not self.master:
            self.value.copy_(self.master)


class Model:
    def __init__(self, vocab=8192, dim=768, hidden=2816, blocks=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale

        self.vocab, self.dim, self.blocks = vocab, dim, blocks
        self.embedding = normal(vocab, dim, scale=1.0).to(BF16)
        # the bank: W_up of block i is matrix 2i, W_down^T is matrix 2i + 1
        g = 2 * blocks
        self.bank = normal(g, hidden, dim, scale=dim ** -0.5).to(BF16)
        self.bank[1::2] *= 0.1
        self.mantissa = torch.zeros(g, hidden, dim, device="cuda", dtype=torch.int16)
        self.grad = torch.zeros(g, hidden, dim, device="cuda")
        self.velocity = torch.zeros(2, g, hidden, dim, device="cuda")
        self.update = torch.empty(g, hidden, dim, device="cuda", dtype=BF16)
        self.energy = torch.zeros(g, max(hidden, dim), device="cuda")
        self.bank_lr = torch.empty(g, device="cuda")
        shape = [(g, hidden, dim)]
        self.link = anvil.alloc_tail_link((g, hidden, dim))
        self.workspace = anvil.alloc_workspace(shape)
        self.tail_workspace = torch.empty(anvil.tail_workspace_bytes(shape), device="cuda", dtype=torch.uint8)
        self.gains = [Adam(torch.ones(dim, device="cuda")) for _ in range(blocks + 1)]
        self.shifts = [Adam(torch.zeros(dim, device="cuda")) for _ in range(blocks + 1)]
        self.head = Adam(normal(vocab, dim, scale=dim ** -0.5), BF16)

    def up(self, i):
        return self.bank[2 * i]

    def down(self, i):
        return self.bank[2 * i + 1].t()

    def forward(self, tokens, save=None):
        """Logits of the next tokens; save: a list that takes what the backward pass needs."""
        x = self.embedding[tokens]
        for i in range(self.blocks):
            h, mean, rstd = anvil.layernorm_forward(x, self.gains[i].value, self.shifts[i].value)
            if save is None:
                a = anvil.linear_forward(h, self.up(i), activation="relu2")
            else:
                a, z = anvil.linear_forward(h, self.up(i), activation="relu2", save_preact=True)
                save.append((x, mean, rstd, h, z, a))
            x = anvil.linear_forward(a, self.down(i), residual=x)
        h, mean, rstd = anvil.layernorm_forward(x, self.gains[-1].value, self.shifts[-1].value)
        if save is not None:
            save.append((x, mean, rstd, h))
        return anvil.linear_forward(h, self.head.value)

    def loss_and_gradients(self, tokens, targets):
        """(loss, entropy) and the gradients: the bank's in self.grad, the others returned as
        (head, [(gain, shift) per norm])."""
        save = []
        logits = self.forward(tokens, save)
        logprob, entropy, lse, _, _ = anvil.token_logprobs(logits, targets)
        seed = torch.full_like(lse, -1.0 / targets.numel())
        dlogits = anvil.token_logprobs_backward(logits, targets, lse, seed, out=logits)
        x, mean, rstd, h = save.pop()
        dh, dhead, _ = anvil.linear_backward(dlogits, h, self.head.value, bias_grad=False, dweight_dtype=F32)
        dx, *norm = anvil.layernorm_backward(dh, x, mean, rstd, self.gains[-1].value, out=dh)
        norms = [tuple(norm)]
        for i in reversed(range(self.blocks)):
            x, mean, rstd, h, z, a = save.pop()
            da, _, _ = anvil.linear_backward(dx, a, self.down(i), bias_grad=False, dweight_dtype=F32,
                                             dweight=self.grad[2 * i + 1].t())
            dh, _, _ = anvil.linear_backward(da, h, self.up(i), preact=z, activation="relu2", bias_grad=False,
                                             dweight_dtype=F32, dweight=self.grad[2 * i])
            dx, *norm = anvil.layernorm_backward(dh, x, mean, rstd, self.gains[i].value, residual_grad=dx, out=dh)
            norms.append(tuple(norm))
        return (-logprob.mean(), entropy.mean()), (dhead, norms[::-1])

    def step(self, tokens, targets, bank_lr=0.01, lr=2e-3):
        """One training step; returns (loss, entropy) as they were before it."""
        stats, (dhead, norms) = self.loss_and_gradients(tokens, targets)
        anvil.multi_bank_step([anvil.Bank(self.grad, self.velocity, self.update, tail_link=self.link)], self.workspace)
        self.bank_lr.fill_(bank_lr)
        anvil.update_tail([anvil.Tail(self.update, self.velocity, self.energy, self.bank, self.mantissa, self.bank_lr,
                                      eff_wd=0.0, beta2=0.95, tail_link=self.link)], self.tail_workspace)
        self.head.update(dhead, lr)
        for (gain, shift), dgain, dshift in zip(zip(self.gains, self.shifts), *zip(*norms)):
            gain.update(dgain, lr)
            shift.update(dshift, lr)
        return stats

    def generate(self, token, count, top=4):
        """`count` tokens after `token`, one call at a time: [(token, its alternatives)] with
        the alternatives as (token, log probability)."""
        out, tokens = [], torch.tensor([token], device="cuda")
        for _ in range(count):
            _, _, _, value, index = anvil.token_logprobs(self.forward(tokens), top=top)
            tokens = index[:, 0].long()
            out.append((int(tokens), list(zip(index[0].tolist(), value[0].tolist()))))
        return out


class Data:
    """Tokens and their successors: `follow[token]` nine times in ten, else any."""

    def __init__(self, vocab, seed=1):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab = vocab
        self.follow = torch.randperm(vocab, generator=self.gen, device="cuda")

    def batch(self, count):
        tokens = torch.randint(0, self.vocab, (count,), generator=self.gen, device="cuda")
        any_token = torch.randint(0, self.vocab, (count,), generator=self.gen, device="cuda")
        usual = torch.rand(count, generator=self.gen, device="cuda") < 0.9
        return tokens, torch.where(usual, self.follow[tokens], any_token)


def train(model, data, steps, tokens, report=None):
    """Trains for `steps` batches of `tokens`; returns the losses."""
    losses = []
    for i in range(steps):
        loss, entropy = model.step(*data.batch(tokens))
        losses.append(loss)
        if report and (i % 10 == 0 or i == steps - 1):
            report(f"step {i:4d}  loss {float(loss):.4f}  entropy {float(entropy):.4f}")
    status = anvil.last_device_error()
    if status != anvil.OK:
        raise RuntimeError(f"device error {anvil.STATUS[status]}")
    return [float(v) for v in losses]


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=16384, help="tokens per step")
    p.add_argument("--vocab", type=int, default=8192)
    p.add_argument("--dim", type=int, default=768)
    p.add_argument("--hidden", type=int, default=2816)
    p.add_argument("--blocks", type=int, default=2)
    a = p.parse_args(argv)
    model, data = Model(a.vocab, a.dim, a.hidden, a.blocks), Data(a.vocab)
    train(model, data, a.steps, a.tokens, report=print)
    token = 17 % a.vocab
    for following, best in model.generate(token, 4):
        print(f"{token} -> {following} (usually {int(data.follow[token])}); "
              + "  ".join(f"{t}: {v:.3f}" for t, v in best))
        token = following


if __name__ == "__main__":
    main()
