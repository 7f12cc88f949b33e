"""Cases of the training-block operators: layer norm, the linear layer with its fused epilogue, and
token log probabilities, each forward and backward, in a plain form of elementary torch operations
(32 bits, rounded once) and through the library (``polynomial_matrix_whitening_gb300.anvil``)."""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5

# the most work of a drawn case: that of the largest listed one of its kind
NORM_ELEMS = 32768 * 2816
LINEAR_FLOPS = 2 * 16384 * 4096 * 16384
LOGPROB_ELEMS = 8192 * 50304


def listed():
    return [
        # the norm before a projection while one token is generated (the 768-wide stream)
        dict(name="norm_token", op="norm", back=False, rows=1, width=768, dtype="bf16", residual=False, pad=0),
        # a norm of an odd width over a ragged batch, rows of a wider buffer
        dict(name="norm_forward_odd", op="norm", back=False, rows=5001, width=1023, dtype="f16", residual=False, pad=1),
        # the backward pass over a hidden layer of a training batch, with the residual's gradient joined in
        dict(name="norm_backward", op="norm", back=True, rows=32768, width=2816, dtype="bf16", residual=True, pad=0),
        # the up projection while one token is generated
        dict(name="linear_token", op="linear", back=False, rows=1, n=2816, k=768, dtype="bf16", act="relu2",
             bias=True, residual=False, transposed=False, grad32=False, pad=0),
        # a ragged prompt through a layer with odd sizes
        dict(name="linear_forward_odd", op="linear", back=False, rows=1000, n=2815, k=771, dtype="f16", act="gelu",
             bias=True, residual=True, transposed=False, grad32=False, pad=0),
        # the up projection's backward pass in a training batch of the mlp bank's layer
        dict(name="linear_backward", op="linear", back=True, rows=8192, n=2816, k=768, dtype="bf16", act="relu2",
             bias=True, residual=False, transposed=False, grad32=False, pad=0),
        # a large model's down projection, its weight held as the transpose, as a bank of one shape holds it
        dict(name="linear_forward_large", op="linear", back=False, rows=16384, n=4096, k=16384, dtype="bf16",
             act="none", bias=True, residual=True, transposed=True, grad32=False, pad=0),
        # a large square layer's backward pass with the weight's gradient in fp32, as the bank step takes it
        dict(name="linear_backward_large", op="linear", back=True, rows=16384, n=4096, k=4096, dtype="bf16",
             act="none", bias=True, residual=False, transposed=False, grad32=True, pad=0),
        # one generated token's log probability and alternatives
        dict(name="logprob_token", op="logprob", back=False, rows=1, vocab=50304, dtype="bf16", top=8, masked=False),
        # scoring a prompt with constrained (masked) tokens, fp32 logits, an odd vocabulary
        dict(name="logprob_forward_odd", op="logprob", back=False, rows=777, vocab=50257, dtype="f32", top=20, masked=True),
        # the loss of a training batch
        dict(name="logprob_forward", op="logprob", back=False, rows=4096, vocab=50304, dtype="bf16", top=0, masked=False),
        # its gradient, with an entropy term
        dict(name="logprob_backward", op="logprob", back=True, rows=8192, vocab=50304, dtype="bf16", top=0, masked=False),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _size(rng, lo, hi):
    """Spread over the logarithm; two in three rounded to what layers usually have, the rest left odd."""
    v = _log_int(rng, lo, hi)
    unit = rng.choice([1, 8, 64])
    return min(hi, max(lo, v // unit * unit or v))


def draw(rng):
    op = rng.choice(["norm", "linear", "logprob"])
    back = rng.random() < 0.5
    if op == "norm":
        width = _size(rng, 16, 16384)
        rows = _log_int(rng, 1, max(1, min(65536, NORM_ELEMS // width)))
        return dict(op=op, back=back, rows=rows, width=width, dtype=rng.choice(["bf16", "f16", "f32"]),
                    residual=back and rng.random() < 0.5, pad=rng.choice([0, 0, 1, 8]))
    if op == "linear":
        n, k = _size(rng, 64, 16384), _size(rng, 64, 16384)
        rows = _log_int(rng, 1, max(1, min(32768, LINEAR_FLOPS // (2 * n * k) // (2 if back else 1))))
        act = rng.choice(["none", "relu2", "gelu", "silu"])
        return dict(op=op, back=back, rows=rows, n=n, k=k, dtype=rng.choice(["bf16", "f16"]), act=act,
                    bias=rng.random() < 0.75, residual=(not back) and rng.random() < 0.5,
                    transposed=rng.random() < 0.5, grad32=back and act == "none", pad=rng.choice([0, 0, 1, 8]))
    vocab = _size(rng, 256, 131072)
    rows = _log_int(rng, 1, max(1, min(16384, LOGPROB_ELEMS // vocab // (1 if back else 2))))
    return dict(op=op, back=back, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "f16", "f32"]),
                top=0 if back else rng.choice([0, 1, 8, 20]), masked=rng.random() < 0.5)


def _randn(shape, gen, scale=1.0, dtype=torch.float32, pad=0):
    """Normal values; with pad, rows of a buffer that is `pad` columns wider."""
    full = tuple(shape[:-1]) + (shape[-1] + pad,)
    t = torch.randn(full, generator=gen, device="cuda").mul_(scale).to(dtype)
    return t[..., :shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPE[case["dtype"]]
    if case["op"] == "norm":
        rows, width, pad = case["rows"], case["width"], case["pad"]
        s = dict(x=_randn((rows, width), gen, 1.5, dt, pad).add_(0.25), w=1.0 + _randn((width,), gen, 0.1), b=_randn((width,), gen, 0.1))
        if case["back"]:
            s["dy"] = _randn((rows, width), gen, 0.1, dt, pad)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
            s["dres"] = _randn((rows, width), gen, 0.1, dt, pad) if case["residual"] else None
    elif case["op"] == "linear":
        rows, n, k, pad = case["rows"], case["n"], case["k"], case["pad"]
        w = _randn((k, n) if case["transposed"] else (n, k), gen, k ** -0.5, dt)
        s = dict(x=_randn((rows, k), gen, 1.0, dt, pad), w=w.t() if case["transposed"] else w,
                 b=_randn((n,), gen, 0.1, dt) if case["bias"] else None)
        if case["back"]:
            s["dy"] = _randn((rows, n), gen, 0.1, dt, pad)
            s["z"] = _randn((rows, n), gen, 1.0, dt) if case["act"] != "none" else None
        else:
            s["r"] = _randn((rows, n), gen, 1.0, dt, pad) if case["residual"] else None
    else:
        rows, vocab = case["rows"], case["vocab"]
        x = _randn((rows, vocab), gen, 2.5)
        if case["masked"]:  # tokens that a grammar or a padded vocabulary forbids; a few rows allow nothing
            x.masked_fill_(torch.rand((rows, vocab), generator=gen, device="cuda") < 0.3, -math.inf)
            x[rows // 2::101] = -math.inf
        s = dict(x=x.to(dt), t=torch.randint(0, vocab, (rows,), generator=gen, device="cuda"))
        if rows > 8:
            s["t"][::17] = -1  # positions that do not count
        if case["back"]:
            xf = s["x"].float()
            s["lse"], s["ent"] = _row_stats(xf)
            live = (s["t"] >= 0).float()
            scale = (2048.0 if case["dtype"] == "f16" else 1.0) / max(1, rows)  # the mean; fp16 with a loss scale
            s["gl"], s["gh"] = -scale * live, 0.01 * scale * live
    s["case"] = case
    return s


# ---------------------------------------------------------------- the plain form
def _act(z, kind):
    if kind == "none":
        return z
    if kind == "relu2":
        return z.clamp_min(0).square()
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z))  # silu


def _act_grad(z, kind):
    if kind == "relu2":
        return 2 * z.clamp_min(0)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


def _row_stats(xf):
    """lse and entropy of each row; a row with no finite logit has lse -inf and entropy 0."""
    m = xf.amax(1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    d = xf - m0
    e = torch.exp(d)
    s = e.sum(1)
    t = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1)
    lse = torch.where(s > 0, m0[:, 0] + torch.log(s), torch.full_like(s, -math.inf))
    ent = torch.where(s > 0, torch.log(s) - t / s, torch.zeros_like(s))
    return lse, ent


def _top(xf, k):
    """The k largest of each row, ties to the lowest index: their order as one 64-bit key."""
    bits = (xf + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) << 32
    key |= xf.shape[1] - 1 - torch.arange(xf.shape[1], device=xf.device)
    got = torch.topk(key, k, dim=1, sorted=True).values
    return (xf.shape[1] - 1 - (got & 0xFFFFFFFF)).to(torch.int32)


def _plain_norm(s, case):
    x = s["x"].float()
    dt = s["x"].dtype
    if not case["back"]:
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
        return (c * rstd[:, None] * s["w"] + s["b"]).to(dt), mean, rstd
    dy = s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"]
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(dt), (dy * xhat).sum(0), dy.sum(0)


def _plain_linear(s, case):
    x, w, dt = s["x"].float(), s["w"].float(), s["x"].dtype
    if not case["back"]:
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return (y.to(dt), z.to(dt)) if case["act"] != "none" else (y.to(dt),)
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), case["act"])
    dw = dz.t() @ x
    return ((dz @ w).to(dt), dw if case["grad32"] else dw.to(dt)) + ((dz.sum(0),) if case["bias"] else ())


def _plain_logprob(s, case):
    x, t = s["x"].float(), s["t"]
    live = t >= 0
    if not case["back"]:
        lse, ent = _row_stats(x)
        xt = x.gather(1, t.clamp_min(0)[:, None])[:, 0]
        none = torch.isinf(lse)
        lp = torch.where(none, torch.full_like(lse, -math.inf), xt - torch.where(none, torch.zeros_like(lse), lse))
        out = (torch.where(live, lp, torch.zeros_like(lp)), ent, lse)
        if case["top"]:
            idx = _top(x, case["top"])
            v = x.gather(1, idx.long())
            out += (torch.where(none[:, None], torch.full_like(v, -math.inf), v - torch.where(none, torch.zeros_like(lse), lse)[:, None]), idx)
        return out
    none = torch.isinf(s["lse"])[:, None]
    logp = x - s["lse"][:, None]
    p = torch.where(none, torch.zeros_like(x), torch.exp(logp))
    plogp = torch.where(p > 0, p * (logp + s["ent"][:, None]), torch.zeros_like(p))
    d = -s["gl"][:, None] * p - s["gh"][:, None] * plogp
    hit = torch.where(live & ~none[:, 0], s["gl"], torch.zeros_like(s["gl"]))
    d.scatter_add_(1, t.clamp_min(0)[:, None], hit[:, None])
    return (torch.where(none, torch.zeros_like(d), d).to(s["x"].dtype),)


# ---------------------------------------------------------------- the library's calls
def _own_norm(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    if not case["back"]:
        return anvil.layernorm_forward(s["x"], s["w"], s["b"], EPS)
    return anvil.layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], residual_grad=s["dres"])


def _own_linear(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    if not case["back"]:
        if case["act"] == "none":
            return (anvil.linear_forward(s["x"], s["w"], s["b"], residual=s["r"]),)
        return anvil.linear_forward(s["x"], s["w"], s["b"], activation=case["act"], residual=s["r"], save_preact=True)
    got = anvil.linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=case["act"],
                                bias_grad=case["bias"], dweight_dtype=torch.float32 if case["grad32"] else None)
    return got if case["bias"] else got[:2]


def _own_logprob(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    if not case["back"]:
        got = anvil.token_logprobs(s["x"], s["t"], top=case["top"])
        return got if case["top"] else got[:3]
    return (anvil.token_logprobs_backward(s["x"], s["t"], s["lse"], s["gl"], entropy=s["ent"], grad_entropy=s["gh"]),)


def run(state):
    case = state["case"]
    form = {"norm": (_plain_norm, _own_norm), "linear": (_plain_linear, _own_linear),
            "logprob": (_plain_logprob, _own_logprob)}[case["op"]]
    return form[1 if own else 0](state, case)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        r, d = case["rows"], case["width"]
        if case["back"]:
            return dict(bytes=r * d * e * (4 if case["residual"] else 3) + 8 * r + 12 * d, flops=14 * r * d)
        return dict(bytes=r * d * e * 2 + 8 * r + 8 * d, flops=8 * r * d)
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        act = case["act"] != "none"
        if case["back"]:
            return dict(bytes=e * (m * n * (2 if act else 1) + 2 * m * k + n * k) + n * k * (4 if case["grad32"] else e)
                        + (4 * n if case["bias"] else 0), flops=4 * m * n * k)
        return dict(bytes=e * (m * k + n * k + m * n * (1 + act + case["residual"]) + (n if case["bias"] else 0)),
                    flops=2 * m * n * k)
    r, v = case["rows"], case["vocab"]
    if case["back"]:
        return dict(bytes=2 * r * v * e + 24 * r, flops=8 * r * v)
    return dict(bytes=r * v * e + 20 * r + 8 * r * case["top"], flops=6 * r * v)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "norm":
        x, w = D["x"], D["w"]
        mu = x.sum(1, keepdim=True) / case["width"]
        var = ((x - mu) ** 2).sum(1, keepdim=True) / case["width"]
        if not case["back"]:
            rs = (var + EPS) ** -0.5
            return (x - mu) * rs * w + D["b"], mu[:, 0], rs[:, 0]
        mu, rs, dy = D["mean"][:, None], D["rstd"][:, None], D["dy"]
        h = (x - mu) * rs
        gw = dy * w
        # the projection of the scaled gradient off the row's constant and off its normalised values
        dx = rs * gw - rs / case["width"] * (gw.sum(1, keepdim=True) + h * (gw * h).sum(1, keepdim=True))
        return dx if D["dres"] is None else dx + D["dres"], torch.einsum("rd,rd->d", dy, h), torch.einsum("rd->d", dy)
    if case["op"] == "linear":
        x, w, kind = D["x"], D["w"], case["act"]
        if case["rows"] * case["n"] * case["k"] > 2e12:
            return None
        if not case["back"]:
            z = torch.matmul(x, w.transpose(0, 1))
            z = z if D["b"] is None else z + D["b"]
            y = z if kind == "none" else {"relu2": lambda v: torch.where(v > 0, v * v, 0 * v),
                                          "gelu": lambda v: v * torch.special.ndtr(v),
                                          "silu": lambda v: v * torch.special.expit(v)}[kind](z)
            y = y if D["r"] is None else y + D["r"]
            return (y, z) if kind != "none" else (y,)
        dz = D["dy"]
        if kind != "none":
            z = D["z"]
            if kind == "relu2":
                dz = torch.where(z > 0, 2 * z * dz, 0 * dz)
            elif kind == "gelu":
                dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            else:
                sg = torch.special.expit(z)
                dz = dz * (sg + z * sg * torch.special.expit(-z))
        out = (torch.matmul(dz, w), torch.matmul(dz.transpose(0, 1), x))
        return out + (dz.sum(0),) if case["bias"] else out
    x, t = D["x"], s["t"]
    lse = torch.logsumexp(x, 1)
    dead = torch.isneginf(lse)
    safe = torch.where(dead, torch.zeros_like(lse), lse)
    p = torch.exp(x - safe[:, None])
    if not case["back"]:
        ent = -torch.special.xlogy(p, p).sum(1) * 1.0
        at = t.clamp_min(0)[:, None]
        lp = torch.where(dead, lse, x.gather(1, at)[:, 0] - safe)
        out = (torch.where(t < 0, torch.zeros_like(lp), lp), ent.masked_fill(dead, 0.0), lse)
        if case["top"]:
            out += (torch.topk(x, case["top"], dim=1).values - safe[:, None], None)
        return out
    lse, ent = D["lse"], D["ent"]
    dead = torch.isneginf(lse)
    p = torch.exp(x - torch.where(dead, torch.zeros_like(lse), lse)[:, None]).masked_fill(dead[:, None], 0.0)
    g = -p * D["gl"][:, None] - D["gh"][:, None] * (torch.special.xlogy(p, p) + p * ent[:, None])
    r = torch.nonzero((t >= 0) & ~dead)[:, 0]
    g[r, t[r]] += D["gl"][r]
    return (g,)
