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

Three options exchange a part each for the operator that does it in fewer launches and less memory:

    --gated       a block is x += W_down (silu(W_gate h) * (W_up h)), h = norm(x): both projections in
                  one kernel, three matrices of a block in the bank
    --fused-loss  head and loss as one operator: no logits in training (and no entropy)
    --adamw BITS  the head (bf16 beside the low half of its fp32 value) and the norms in one AdamW
                  step, its moments in 32 or 8 bits

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


class Parameter:
    """A parameter of the AdamW step: `value` in fp32, or in bf16 with the fp32 value's low half beside it."""

    def __init__(self, init, compute=F32, bits=32):
        init, self.mantissa = init.to(F32).contiguous(), None
        self.value = init
        if compute == BF16:
            halves = init.view(torch.int32)
            self.value = (halves >> 16).to(torch.int16).view(BF16)
            self.mantissa = (halves << 16 >> 16).to(torch.int16)
        self.state = anvil.adamw_state(self.value, bits)


def adamw(parameters, grads, step, lr, weight_decay=0.0):
    """One AdamW step of all of them."""
    exp_avgs, exp_avg_sqs, scales = zip(*(p.state for p in parameters))
    anvil.adamw_step([p.value for p in parameters], grads, exp_avgs, exp_avg_sqs, lr, step, weight_decay=weight_decay,
                     mantissas=[p.mantissa for p in parameters], scales=scales)


class Model:
    def __init__(self, vocab=8192, dim=768, hidden=2816, blocks=2, seed=0, gated=False, fused_loss=False, adamw=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale

        self.vocab, self.dim, self.blocks = vocab, dim, blocks
        self.gated, self.fused_loss, self.adamw, self.steps = gated, fused_loss, adamw, 0
        self.embedding = normal(vocab, dim, scale=1.0).to(BF16)
        # the bank: W_up of block i is matrix 2i, W_down^T is matrix 2i + 1; gated: W_gate, W_up, W_down^T
        self.per_block = 3 if gated else 2
        g = self.per_block * blocks
        self.bank = normal(g, hidden, dim, scale=dim ** -0.5).to(BF16)
        self.bank[self.per_block - 1::self.per_block] *= 0.1
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
        vector, matrix = Adam, Adam
        if adamw:  # a norm's moments are small: 32 bits
            vector, matrix = Parameter, lambda init, compute: Parameter(init, compute, adamw)
        self.gains = [vector(torch.ones(dim, device="cuda")) for _ in range(blocks + 1)]
        self.shifts = [vector(torch.zeros(dim, device="cuda")) for _ in range(blocks + 1)]
        self.head = matrix(normal(vocab, dim, scale=dim ** -0.5), BF16)

    def gate(self, i, of=None):
        return (self.bank if of is None else of)[self.per_block * i]

    def up(self, i, of=None):
        return (self.bank if of is None else of)[self.per_block * (i + 1) - 2]

    def down(self, i, of=None):
        return (self.bank if of is None else of)[self.per_block * (i + 1) - 1].t()

    def hidden(self, tokens, save=None):
        """What the head multiplies; save: a list that takes what the backward pass needs."""
        x = self.embedding[tokens]
        for i in range(self.blocks):
            h, mean, rstd = anvil.layernorm_forward(x, self.gains[i].value, self.shifts[i].value)
            if self.gated:
                a = anvil.gated_linear_forward(h, self.gate(i), self.up(i), save_preact=save is not None)
            else:
                a = anvil.linear_forward(h, self.up(i), activation="relu2", save_preact=save is not None)
            if save is not None:
                a, *z = a
                save.append((x, mean, rstd, h, z, a))
            x = anvil.linear_forward(a, self.down(i), residual=x)
        h, mean, rstd = anvil.layernorm_forward(x, self.gains[-1].value, self.shifts[-1].value)
        if save is not None:
            save.append((x, mean, rstd, h))
        return h

    def forward(self, tokens, save=None):
        """Logits of the next tokens; save as hidden's."""
        return anvil.linear_forward(self.hidden(tokens, save), self.head.value)

    def loss_and_gradients(self, tokens, targets):
        """(loss, entropy) and the gradients: the bank's in self.grad, the others returned as
        (head, [(gain, shift) per norm])."""
        save = []
        if self.fused_loss:
            h = self.hidden(tokens, save)
            loss, lse = anvil.linear_cross_entropy(h, self.head.value, targets)
            seed = torch.full_like(lse, 1.0 / targets.numel())
            dh, dhead = anvil.linear_cross_entropy_backward(h, self.head.value, targets, lse, seed, dweight_dtype=F32)
            stats = (loss.mean(), None)
        else:
            logits = self.forward(tokens, save)
            h = save[-1][3]
            logprob, entropy, lse, _, _ = anvil.token_logprobs(logits, targets)
            seed = torch.full_like(lse, -1.0 / targets.numel())
            dlogits = anvil.token_logprobs_backward(logits, targets, lse, seed, out=logits)
            dh, dhead, _ = anvil.linear_backward(dlogits, h, self.head.value, bias_grad=False, dweight_dtype=F32)
            stats = (-logprob.mean(), entropy.mean())
        x, mean, rstd, h = save.pop()
        dx, *norm = anvil.layernorm_backward(dh, x, mean, rstd, self.gains[-1].value, out=dh)
        norms = [tuple(norm)]
        for i in reversed(range(self.blocks)):
            x, mean, rstd, h, z, a = save.pop()
            da, _, _ = anvil.linear_backward(dx, a, self.down(i), bias_grad=False, dweight_dtype=F32,
                                             dweight=self.down(i, self.grad))
            if self.gated:
                dh, _, _ = anvil.gated_linear_backward(da, h, self.gate(i), self.up(i), *z, dweight_dtype=F32,
                                                       dgate=self.gate(i, self.grad), dup=self.up(i, self.grad))
            else:
                dh, _, _ = anvil.linear_backward(da, h, self.up(i), preact=z[0], activation="relu2", bias_grad=False,
                                                 dweight_dtype=F32, dweight=self.up(i, self.grad))
            dx, *norm = anvil.layernorm_backward(dh, x, mean, rstd, self.gains[i].value, residual_grad=dx, out=dh)
            norms.append(tuple(norm))
        return stats, (dhead, norms[::-1])

    def step(self, tokens, targets, bank_lr=0.01, lr=2e-3):
        """One training step; returns (loss, entropy) as they were before it (no entropy with the fused loss)."""
        stats, (dhead, norms) = self.loss_and_gradients(tokens, targets)
        anvil.multi_bank_step([anvil.Bank(self.grad, self.velocity, self.update, tail_link=self.link)], self.workspace)
        self.bank_lr.fill_(bank_lr)
        anvil.update_tail([anvil.Tail(self.update, self.velocity, self.energy, self.bank, self.mantissa, self.bank_lr,
                                      eff_wd=0.0, beta2=0.95, tail_link=self.link)], self.tail_workspace)
        if self.adamw:
            self.steps += 1
            adamw([self.head] + self.gains + self.shifts, [dhead] + [g for g, _ in norms] + [g for _, g in norms],
                  self.steps, lr)
            return stats
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
            report(f"step {i:4d}  loss {float(loss):.4f}" + ("" if entropy is None else f"  entropy {float(entropy):.4f}"))
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
    p.add_argument("--gated", action="store_true", help="gated blocks")
    p.add_argument("--fused-loss", action="store_true", help="head and loss as one operator")
    p.add_argument("--adamw", type=int, choices=(8, 32), help="AdamW for head and norms, its moments in so many bits")
    a = p.parse_args(argv)
    model = Model(a.vocab, a.dim, a.hidden, a.blocks, gated=a.gated, fused_loss=a.fused_loss, adamw=a.adamw)
    data = Data(a.vocab)
    train(model, data, a.steps, a.tokens, report=print)
    token = 17 % a.vocab
    for following, best in model.generate(token, 4):
        print(f"{token} -> {following} (usually {int(data.follow[token])}); "
              + "  ".join(f"{t}: {v:.3f}" for t, v in best))
        token = following


if __name__ == "__main__":
    main()
