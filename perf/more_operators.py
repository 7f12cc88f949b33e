"""Cases of the operators that make up a training step around the banks: the gated projection of a
feed-forward block and the cross entropy of a head without its logits, each forward and backward, and
AdamW over many tensors at once with states in 32 or 8 bits; in a plain form of elementary torch
operations (32 bits, rounded once) and through the library (``polynomial_matrix_whitening_gb300.anvil``)."""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "bf16m": 4}

# the most work of a drawn case: that of the largest listed one of its kind
GATED_FLOPS = 4 * 16384 * 8192 * 4096
HEAD_FLOPS = 6 * 8192 * 50304 * 768
HEAD_LOGITS = 8192 * 50304
ADAMW_COUNT = 1 << 27

# AdamW's constants, and the 8-bit states' blocks: 256 values share a scale
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 7
BLOCK = 256
TOP_M, TOP_R = 448.0, 31.0 * 2 ** 14  # the largest code's value: e4m3, and the unsigned code of the root


def listed():
    return [
        # a block's gated projection while one token is generated
        dict(name="gated_token", op="gated", back=False, rows=1, n=2816, k=768, dtype="bf16", act="silu",
             transposed=False, save=False, pad=0),
        # a ragged prompt through a layer with odd sizes, rows of wider buffers, what the backward pass needs kept
        dict(name="gated_forward_odd", op="gated", back=False, rows=1000, n=2815, k=771, dtype="f16", act="gelu",
             transposed=False, save=True, pad=1),
        # a training batch of the stream's own layer, the gradient in bf16 as the bank step takes it
        dict(name="gated_backward", op="gated", back=True, rows=8192, n=2816, k=768, dtype="bf16", act="silu",
             transposed=False, save=False, pad=0),
        # a large model's layer, its weights held as the transposes
        dict(name="gated_forward_large", op="gated", back=False, rows=16384, n=8192, k=4096, dtype="bf16", act="silu",
             transposed=True, save=False, pad=0),
        # scoring one token
        dict(name="head_token", op="head", back=False, rows=1, vocab=50304, k=768, dtype="bf16", transposed=False,
             pad=0),
        # scoring a prompt, an odd vocabulary, a third of the positions not counted
        dict(name="head_forward_odd", op="head", back=False, rows=777, vocab=50257, k=771, dtype="f16",
             transposed=False, pad=1),
        # the loss of a training batch
        dict(name="head_forward", op="head", back=False, rows=8192, vocab=50304, k=768, dtype="bf16",
             transposed=False, pad=0),
        # its gradient, the head's in bf16 as the optimizer takes it
        dict(name="head_backward", op="head", back=True, rows=8192, vocab=50304, k=768, dtype="bf16",
             transposed=False, pad=0),
        # the gains and shifts of a few norms: one small launch
        dict(name="adamw_vectors", op="adamw", tensors=6, count=6 * 768, param="f32", grad="f32", bits=32, odd=False),
        # bf16 weights that keep their fp32 master's low half, bf16 gradients, states in 32 bits
        dict(name="adamw_master", op="adamw", tensors=100, count=50000000, param="bf16m", grad="bf16", bits=32, odd=False),
        # tensors of a flat buffer, one after the other with odd sizes, states in 8 bits
        dict(name="adamw_8bit_odd", op="adamw", tensors=37, count=3000001, param="bf16", grad="bf16", bits=8, odd=True),
        # a model's fp32 weights and gradients with states in 8 bits
        dict(name="adamw_8bit", op="adamw", tensors=200, count=1 << 27, param="f32", grad="f32", bits=8, odd=False),
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
    op = rng.choice(["gated", "head", "adamw"])
    back = rng.random() < 0.5
    if op == "gated":
        n, k = _size(rng, 64, 16384), _size(rng, 64, 8192)
        rows = _log_int(rng, 1, max(1, min(32768, GATED_FLOPS // (4 * n * k) // (2 if back else 1))))
        return dict(op=op, back=back, rows=rows, n=n, k=k, dtype=rng.choice(["bf16", "f16"]),
                    act=rng.choice(["silu", "gelu", "gelu_tanh", "relu2", "none"]), transposed=rng.random() < 0.5,
                    save=not back and rng.random() < 0.5, pad=rng.choice([0, 0, 1, 8]))
    if op == "head":
        vocab, k = _size(rng, 256, 131072), _size(rng, 64, 4096)
        rows = _log_int(rng, 1, max(1, min(16384, HEAD_FLOPS // (2 * vocab * k) // (3 if back else 1), HEAD_LOGITS // vocab)))
        return dict(op=op, back=back, rows=rows, vocab=vocab, k=k, dtype=rng.choice(["bf16", "f16"]),
                    transposed=rng.random() < 0.25, pad=rng.choice([0, 0, 1, 8]))
    tensors = _log_int(rng, 1, 400)
    param = rng.choice(["f32", "bf16", "f16", "bf16m"])
    return dict(op=op, tensors=tensors, count=_log_int(rng, 64 * tensors, ADAMW_COUNT), param=param,
                grad="f32" if param == "f32" and rng.random() < 0.5 else rng.choice(["bf16", "f32"]) if param != "f16" else "f16",
                bits=rng.choice([8, 32]), odd=rng.random() < 0.4)


def _randn(shape, gen, scale=1.0, dtype=torch.float32, pad=0):
    """Normal values; with pad, rows of a buffer that is `pad` columns wider."""
    full = tuple(shape[:-1]) + (shape[-1] + pad,)
    t = torch.randn(full, generator=gen, device="cuda").mul_(scale).to(dtype)
    return t[..., :shape[-1]]


def _weight(n, k, transposed, gen, scale, dt):
    w = _randn((k, n) if transposed else (n, k), gen, scale, dt)
    return w.t() if transposed else w


def _sizes(case):
    """The tensors' sizes, fixed by the case: a few large ones and many small, as a model has them."""
    n, total = case["tensors"], case["count"]
    share = [1.0 / (1 + (i * 7) % n) for i in range(n)]
    out = [max(1, int(total * s / sum(share))) for s in share]
    if not case["odd"]:  # whole blocks of 64, as widths have them
        out = [max(64, s // 64 * 64) for s in out]
    return out


def _views(flat, sizes, step):
    """Tensors of those sizes in a flat buffer, each on the next multiple of `step`."""
    out, at = [], 0
    for s in sizes:
        out.append(flat[at:at + s])
        at += -(-s // step) * step
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    dt, rows, k, pad = DTYPE[case["dtype"]], case["rows"], case["k"], case["pad"]
    s = dict(case=case)
    if case["op"] == "gated":
        n = case["n"]
        s["x"] = _randn((rows, k), gen, 1.0, dt, pad)
        s["wg"], s["wu"] = (_weight(n, k, case["transposed"], gen, k ** -0.5, dt) for _ in range(2))
        if case["back"]:
            s["dy"] = _randn((rows, n), gen, 0.1, dt, pad)
            s["g"], s["u"] = _randn((rows, n), gen, 1.0, dt), _randn((rows, n), gen, 1.0, dt)
        return s
    vocab = case["vocab"]
    s["x"] = _randn((rows, k), gen, 1.0, dt, pad)
    s["w"] = _weight(vocab, k, case["transposed"], gen, 2.0 * k ** -0.5, dt)
    s["t"] = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    if rows > 8:
        s["t"][::3] = -1  # positions that do not count
    if case["back"]:
        s["lse"] = torch.empty(rows, device="cuda")
        wf = s["w"].double() if rows * vocab * k < 1e10 else s["w"].float()
        for r in range(0, rows, 1024):
            s["lse"][r:r + 1024] = torch.logsumexp(s["x"][r:r + 1024].to(wf.dtype) @ wf.t(), 1).float()
        s["gl"] = torch.full((rows,), 1.0 / rows, device="cuda")  # the mean
    return s


def _prepare_adamw(case, gen):
    sizes = _sizes(case)
    step = 1 if case["odd"] else 64
    total = sum(-(-z // step) * step for z in sizes)
    s = dict(case=case, sizes=sizes, step=step)
    master = _randn((total,), gen, 0.05)
    if case["param"] == "bf16m":  # the high half, and the low half beside it
        bits = master.view(torch.int32)
        s["flat_p"] = (bits >> 16).to(torch.int16).view(torch.bfloat16)
        s["flat_low"] = (bits << 16 >> 16).to(torch.int16)
        s["low"] = _views(s["flat_low"], sizes, step)
    else:
        s["flat_p"] = master.to(DTYPE[case["param"]])
        s["low"] = None
    s["flat_g"] = _randn((total,), gen, 0.01, DTYPE[case["grad"]])
    m = _randn((total,), gen, 0.004)
    v = _randn((total,), gen, 0.01).square_()
    s["p"], s["g"] = _views(s["flat_p"], sizes, step), _views(s["flat_g"], sizes, step)
    if case["bits"] == 32:
        s["flat_m"], s["flat_v"], s["scales"] = m, v, None
    else:
        s["flat_m"] = torch.zeros(total, device="cuda", dtype=torch.float8_e4m3fn)
        s["flat_v"] = torch.zeros(total, device="cuda", dtype=torch.uint8)
        blocks = [-(-z // BLOCK) for z in sizes]
        s["flat_scales"] = torch.zeros(2 * sum(blocks), device="cuda")
        s["scales"] = [f.view(2, -1) for f in torch.split(s["flat_scales"], [2 * b for b in blocks])]
        s["out_m"], s["out_v"] = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
        s["out"] = (_views(s["out_m"], sizes, step), _views(s["out_v"], sizes, step))
    s["m"], s["v"] = _views(s["flat_m"], sizes, step), _views(s["flat_v"], sizes, step)
    if case["bits"] == 8:
        for mi, vi, m8, v8, sc in zip(_views(m, sizes, step), _views(v, sizes, step), s["m"], s["v"], s["scales"]):
            _pack(mi, torch.sqrt(vi), m8, v8, sc)
    return s


# ---------------------------------------------------------------- the plain form
def _act(z, kind):
    if kind == "none":
        return z
    if kind == "relu2":
        return z.clamp_min(0).square()
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))  # silu


def _act_grad(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu2":
        return 2 * z.clamp_min(0)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        sg = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return sg + z * sg * (1 - sg) * c * (1 + 3 * 0.044715 * z * z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


def _plain_gated(s, case):
    x, wg, wu, dt, kind = s["x"].float(), s["wg"].float(), s["wu"].float(), s["x"].dtype, case["act"]
    if not case["back"]:
        g, u = x @ wg.t(), x @ wu.t()
        y = (_act(g, kind) * u).to(dt)
        return (y, g.to(dt), u.to(dt)) if case["save"] else (y,)
    g, u, dy = s["g"].float(), s["u"].float(), s["dy"].float()
    dg, du = dy * u * _act_grad(g, kind), dy * _act(g, kind)
    return (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)


def _plain_head(s, case):
    x, w, t, dt = s["x"].float(), s["w"].float(), s["t"], s["x"].dtype
    live = t >= 0
    z = x @ w.t()
    if not case["back"]:
        m = z.amax(1)
        lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
        loss = lse - z.gather(1, t.clamp_min(0)[:, None])[:, 0]
        return torch.where(live, loss, torch.zeros_like(loss)), lse
    gl = torch.where(live, s["gl"], torch.zeros_like(s["gl"]))
    d = torch.exp(z - s["lse"][:, None])
    d[torch.arange(t.numel(), device=t.device), t.clamp_min(0)] -= 1.0
    d *= gl[:, None]
    return (d @ w).to(dt), (d.t() @ x).to(dt)


def _blocks(t):
    """A flat tensor as rows of one block each, the last one filled with zeros."""
    n = t.numel()
    return torch.cat([t, t.new_zeros(-n % BLOCK)]).view(-1, BLOCK)


def _root_values(code):
    """0 to 15 as they are, then 16 steps in each doubling."""
    c = code.int()
    return torch.where(c < 16, c, (16 + (c & 15)) << ((c >> 4) - 1).clamp_min(0)).float()


def _root_codes(q):
    """The nearest code of q >= 0, ties to the even one; what is not 0 stays above it."""
    bits = q.view(torch.int32)
    big = ((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) - (131 << 4) + 16
    code = torch.where(q < 16, torch.round(q).int(), big)
    return torch.where(q > 0, code.clamp(1, 255), torch.zeros_like(code))


def _pack(m, r, m8, r8, scales):
    """The first moment and the second one's root into 8-bit codes and one scale a block."""
    mb, rb, n = _blocks(m), _blocks(r), m.numel()
    for i, (b, top) in enumerate(((mb, TOP_M), (rb, TOP_R))):
        most = b.abs().amax(1)
        most = torch.where(most < 2.0 ** -100, torch.zeros_like(most), most)
        inverse = torch.where(most > 0, torch.full_like(most, top) / most, torch.zeros_like(most))
        scales[i] = most * (1.0 / top)
        q = b * inverse[:, None]
        if i:
            r8.copy_(_root_codes(q).to(torch.uint8).view(-1)[:n])
        else:
            m8.copy_(q.to(torch.float8_e4m3fn).view(-1)[:n])


def _unpack(m8, r8, scales):
    n = m8.numel()
    m = _blocks(m8.float()) * scales[0][:, None]
    r = _blocks(_root_values(r8)) * scales[1][:, None]
    return m.view(-1)[:n], r.view(-1)[:n]


def _constants():
    return dict(step_size=LR / (1 - BETA1 ** STEP), root=1 / math.sqrt(1 - BETA2 ** STEP), decay=1 - LR * DECAY)


def _plain_adamw(s, case):
    k = _constants()
    for i, (p, g) in enumerate(zip(s["p"], s["g"])):
        if case["param"] == "bf16m":
            x = ((p.view(torch.int16).int() << 16) | (s["low"][i].int() & 0xFFFF)).view(torch.float32)
        else:
            x = p.float()
        g = g.float()
        if case["bits"] == 8:
            m, r = _unpack(s["m"][i], s["v"][i], s["scales"][i])
            v = r * r
        else:
            m, v = s["m"][i], s["v"][i]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * (1 - BETA2)) * g
        r = torch.sqrt(v)
        x = x * k["decay"] - (m / (r * k["root"] + EPS)) * k["step_size"]
        if case["param"] == "bf16m":
            bits = x.view(torch.int32)
            p.copy_((bits >> 16).to(torch.int16).view(torch.bfloat16))
            s["low"][i].copy_((bits << 16 >> 16).to(torch.int16))
        else:
            p.copy_(x)
        if case["bits"] == 8:
            _pack(m, r, s["m"][i], s["v"][i], s["scales"][i])
            m, r = _unpack(s["m"][i], s["v"][i], s["scales"][i])
            s["out"][0][i].copy_(m)
            s["out"][1][i].copy_(r * r)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    return _adamw_outputs(s, case)


def _adamw_outputs(s, case):
    out = (s["flat_p"],) + ((s["out_m"], s["out_v"]) if case["bits"] == 8 else (s["flat_m"], s["flat_v"]))
    return out + ((s["flat_low"],) if case["param"] == "bf16m" else ())


# ---------------------------------------------------------------- the library's calls
def _own_gated(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    if not case["back"]:
        got = anvil.gated_linear_forward(s["x"], s["wg"], s["wu"], activation=case["act"], save_preact=case["save"])
        return got if case["save"] else (got,)
    return anvil.gated_linear_backward(s["dy"], s["x"], s["wg"], s["wu"], s["g"], s["u"], activation=case["act"])


def _own_head(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    if not case["back"]:
        return anvil.linear_cross_entropy(s["x"], s["w"], s["t"])
    return anvil.linear_cross_entropy_backward(s["x"], s["w"], s["t"], s["lse"], s["gl"])


def _own_adamw(s, case):
    from polynomial_matrix_whitening_gb300 import anvil
    anvil.adamw_step(s["p"], s["g"], s["m"], s["v"], LR, STEP, BETA1, BETA2, EPS, DECAY, mantissas=s["low"],
                     scales=s["scales"])
    if case["bits"] == 8:
        anvil.adamw_values(s["m"], s["v"], s["scales"], out=s["out"])
    return _adamw_outputs(s, case)


def run(state):
    case = state["case"]
    form = {"gated": (_plain_gated, _own_gated), "head": (_plain_head, _own_head),
            "adamw": (_plain_adamw, _own_adamw)}[case["op"]]
    return form[1 if own else 0](state, case)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK  # 8 bits: and the values that it stands for
        return dict(bytes=int(n * (2 * SIZE[case["param"]] + SIZE[case["grad"]] + state)), flops=16 * n)
    e, r, k = SIZE[case["dtype"]], case["rows"], case["k"]
    n = case["n"] if case["op"] == "gated" else case["vocab"]
    if case["op"] == "gated":
        if case["back"]:
            return dict(bytes=e * (3 * r * n + 2 * r * k + 4 * n * k), flops=8 * r * n * k)
        return dict(bytes=e * (r * k + 2 * n * k + (3 if case["save"] else 1) * r * n), flops=4 * r * n * k)
    if case["back"]:  # the logits are not kept: their product is part of the gradient
        return dict(bytes=e * (2 * r * k + 2 * n * k) + 16 * r, flops=6 * r * n * k)
    return dict(bytes=e * (r * k + n * k) + 16 * r, flops=2 * r * n * k)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_act(z, kind):
    """Value and slope."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu2":
        return torch.where(z > 0, z * z, 0 * z), torch.where(z > 0, 2 * z, 0 * z)
    if kind == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z ** 3))
        return z * (1 + th) / 2, (1 + th) / 2 + z / 2 * (1 - th * th) * c * (1 + 0.134145 * z * z)
    sg = torch.special.expit(z)
    return z * sg, sg + z * sg * torch.special.expit(-z)


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    k = _constants()
    p, m_out, v_out = s["flat_p"].double(), s["flat_m"].double(), s["flat_v"].double()
    at = 0
    for i, n in enumerate(s["sizes"]):
        g = s["g"][i].double()
        if case["param"] == "bf16m":
            x = ((s["p"][i].view(torch.int16).int() << 16) | (s["low"][i].int() & 0xFFFF)).view(torch.float32).double()
        else:
            x = s["p"][i].double()
        if case["bits"] == 32:
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            reach = torch.arange(n, device="cuda") // BLOCK
            m = s["m"][i].float().double() * s["scales"][i][0].double()[reach]
            c = s["v"][i].long()
            root = torch.where(c < 16, c, (16 + c % 16) * 2 ** (c // 16 - 1).clamp_min(0)).double()
            v = (root * s["scales"][i][1].double()[reach]) ** 2
        m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g ** 2
        p[at:at + n] = k["decay"] * x - k["step_size"] * m / (v.sqrt() * k["root"] + EPS)
        m_out[at:at + n], v_out[at:at + n] = m, v
        at += -(-n // s["step"]) * s["step"]
    if case["param"] == "bf16m":  # both halves of the fp32 value are bits of it, not numbers near one
        p = None
    if case["bits"] == 8:  # next to a border between two codes either one is right
        m_out = v_out = None
    return p, m_out, v_out


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    n = case["n"] if case["op"] == "gated" else case["vocab"]
    if (2 if case["op"] == "gated" else 1) * (3 if case["back"] else 1) * case["rows"] * n * case["k"] > 2e12:
        return None
    s = prepare(case, seed)
    D = {key: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for key, v in s.items()}
    x = D["x"]
    if case["op"] == "gated":
        if not case["back"]:
            g, u = torch.einsum("rk,nk->rn", x, D["wg"]), torch.einsum("rk,nk->rn", x, D["wu"])
            y = _exact_act(g, case["act"])[0] * u
            return (y, g, u) if case["save"] else (y,)
        value, slope = _exact_act(D["g"], case["act"])
        dg, du = D["dy"] * slope * D["u"], D["dy"] * value
        return (torch.einsum("rn,nk->rk", dg, D["wg"]) + torch.einsum("rn,nk->rk", du, D["wu"]),
                torch.einsum("rn,rk->nk", dg, x), torch.einsum("rn,rk->nk", du, x))
    z, t = torch.einsum("rk,vk->rv", x, D["w"]), s["t"]
    if not case["back"]:
        lse = torch.logsumexp(z, 1)
        return torch.where(t < 0, torch.zeros_like(lse), lse - z.gather(1, t.clamp_min(0)[:, None])[:, 0]), lse
    gl = D["gl"].masked_fill(t < 0, 0.0)
    hot = torch.zeros_like(z).scatter_(1, t.clamp_min(0)[:, None], 1.0)
    d = (torch.exp(z - D["lse"][:, None]) - hot) * gl[:, None]
    return torch.einsum("rv,vk->rk", d, D["w"]), torch.einsum("rv,rk->vk", d, x)
