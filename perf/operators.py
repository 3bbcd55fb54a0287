"""Cases that measure the gated linear recurrence and the gated group norm.

Each case is one pass a user makes: a prefill (``scan_fwd``), a training step's forward and
backward (``scan_train``, ``norm_train``), one token for every session and layer
(``scan_step``) or a normalised, gated read-out (``norm_fwd``).  ``run`` computes it in plain
torch operations, or, with ``own`` set, through the package's entry points.  In the step case
B x T is sessions x layers and the state is updated in place, as a decode loop does.

    recurrence   f = sigma(g), i = 1 - f:  h_t = f_t h_{t-1} + i_t x_t,  y_t = h_t
    group norm   n = (x - mean) / sqrt(var + eps) per row and group,  a = n weight + bias,
                 y = a act(z), or act(a) without z
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 64e-5


def listed():
    return [
        # the shortest prompt of a small model: launch and latency
        dict(name="scan_fwd_1x64x64", op="scan_fwd", B=1, T=64, C=64, dtype="f32"),
        # a batch of prompts continued from stored states
        dict(name="scan_fwd_8x1024x768", op="scan_fwd", B=8, T=1024, C=768, dtype="f32"),
        # one long document: few rows, a long axis
        dict(name="scan_fwd_1x16384x4096", op="scan_fwd", B=1, T=16384, C=4096, dtype="f32"),
        # training steps of a layer, fp32 and bf16
        dict(name="scan_train_8x1024x768", op="scan_train", B=8, T=1024, C=768, dtype="f32"),
        dict(name="scan_train_4x4096x2048_bf16", op="scan_train", B=4, T=4096, C=2048, dtype="bf16"),
        # odd length and width: rows that are not a multiple of 16 bytes
        dict(name="scan_train_3x1001x257_bf16", op="scan_train", B=3, T=1001, C=257, dtype="bf16"),
        # one token: a few sessions of a small model, and a full serving batch of a large one
        dict(name="scan_step_8x12x768_bf16", op="scan_step", B=8, T=12, C=768, dtype="bf16"),
        dict(name="scan_step_256x32x4096", op="scan_step", B=256, T=32, C=4096, dtype="f32"),
        # the read-out of one token for 256 sessions, 64 heads
        dict(name="norm_fwd_256x1x4096", op="norm_fwd", B=256, T=1, C=4096, dtype="f32", groups=64, act="silu", gate=True),
        # training steps of the read-out: 64-channel heads with a SiLU gate
        dict(name="norm_train_8x1024x768", op="norm_train", B=8, T=1024, C=768, dtype="f32", groups=12, act="silu", gate=True),
        dict(name="norm_train_4x4096x2048_bf16", op="norm_train", B=4, T=4096, C=2048, dtype="bf16", groups=32, act="silu", gate=True),
        # odd groups of 65 channels, the activation on the normalised value
        dict(name="norm_train_3x1001x520", op="norm_train", B=3, T=1001, C=520, dtype="f32", groups=8, act="silu", gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_train", "scan_step", "norm_fwd", "norm_train"])
    case = dict(op=op, dtype=rng.choice(["f32", "bf16"]))
    most = 1 << 25
    while True:
        if op == "scan_step":
            case.update(B=_log(rng, 1, 256), T=rng.randint(1, 32), C=_log(rng, 64, 4096))
        elif op.startswith("scan"):
            case.update(B=_log(rng, 1, 16), T=_log(rng, 1, 16384), C=_log(rng, 33, 4096))
        else:
            D = rng.choice([_log(rng, 8, 256), 64, 128, 2 * _log(rng, 4, 1024)])
            G = max(1, _log(rng, 64, 4096) // D)
            case.update(B=_log(rng, 1, 64), T=_log(rng, 1, 4096), C=D * G, groups=G,
                        act=rng.choice(["silu", "sigmoid", "none"]), gate=rng.random() < 0.7)
        if case["B"] * case["T"] * case["C"] <= most:
            return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, T, C, dt = case["B"], case["T"], case["C"], _DT[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    s = dict(case)
    if case["op"].startswith("scan"):
        # gate logits that mostly remember (memories of a few to a few hundred tokens)
        s["g"] = normal(B, T, C, mean=2.0, std=1.5).to(dt)
        s["x"] = normal(B, T, C).to(dt)
        if case["op"] == "scan_step":
            s["state"] = normal(B, T, C)
        else:
            s["state_in"] = normal(B, C)
        if case["op"] == "scan_train":
            s["gy"] = normal(B, T, C).to(dt)
            s["gstate"] = normal(B, C)
    else:
        G = case["groups"]
        # a recurrence's read-out: heads of unlike scale and offset
        x = normal(B, T, G, C // G) * torch.exp(normal(G, 1)) + normal(G, 1, std=0.5)
        s["x"] = x.reshape(B, T, C).to(dt)
        s["z"] = normal(B, T, C).to(dt) if case["gate"] else None
        s["weight"] = normal(C, mean=1.0, std=0.1)
        s["bias"] = normal(C, std=0.1)
        if case["op"] == "norm_train":
            s["gy"] = normal(B, T, C).to(dt)
    return s


def run(s):
    if own:
        return _own(s)
    return _scan(s) if s["op"].startswith("scan") else _norm(s)


def _own(s):
    import linear_attention_rnn_wkv_b200 as wkv
    op = s["op"]
    if op == "scan_step":
        return wkv.gated_scan_step(s["g"], s["x"], s["state"]), s["state"]
    if op == "scan_fwd":
        return wkv.gated_scan_forward(s["g"], s["x"], state_in=s["state_in"])[:2]
    if op == "scan_train":
        y, state_out, carry = wkv.gated_scan_forward(s["g"], s["x"], state_in=s["state_in"], want_carry=True)
        grads = wkv.gated_scan_backward(s["g"], s["x"], carry, s["gy"], gstate_out=s["gstate"])
        if s["gy"].dtype == torch.float32:
            # the plain form leaves the final state's gradient added to an fp32 gy; the next pass on
            # this state has to find the same gy
            s["gy"].select(1, -1).add_(s["gstate"])
        return (y, state_out) + grads
    how = dict(groups=s["groups"], eps=_EPS, act=s["act"])
    y = wkv.group_norm_gated(s["x"], s["z"], s["weight"], s["bias"], **how)
    if op == "norm_fwd":
        return y
    return (y,) + wkv.group_norm_gated_backward(s["x"], s["z"], s["weight"], s["bias"], s["gy"], **how)


# ---- the plain forms (32 bits, rounded to the inputs' type at the end) ----


def _gates(g):
    """(f, 1 - f), each from its own exponential so that neither is a difference."""
    g = g.float()
    return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, in log2(T) doubling steps."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _scan(s):
    x, dt = s["x"].float(), s["x"].dtype
    f, i = _gates(s["g"])
    if s["op"] == "scan_step":
        s["state"].mul_(f).add_(i * x)
        return s["state"].to(dt), s["state"]
    b = i * x
    b[:, 0] += f[:, 0] * s["state_in"]
    h = _linear_scan(f, b)
    out = (h.to(dt), h[:, -1].clone())
    if s["op"] == "scan_fwd":
        return out
    lam = s["gy"].float()
    lam[:, -1] += s["gstate"]
    later = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)
    lam = _linear_scan(later.flip(1), lam.flip(1)).flip(1)
    before = torch.cat([s["state_in"][:, None], h[:, :-1]], 1)
    return out + ((f * i * (before - x) * lam).to(dt), (i * lam).to(dt), f[:, 0] * lam[:, 0])


def _act(v, act):
    """act(v) and its derivative."""
    if act == "none":
        return v, torch.ones_like(v)
    p = 1 / (1 + torch.exp(-v))
    q = 1 / (1 + torch.exp(v))
    return (v * p, p + v * p * q) if act == "silu" else (p, p * q)


def _norm(s):
    dt, G, C = s["x"].dtype, s["groups"], s["C"]
    x = s["x"].float().unflatten(-1, (G, C // G))
    d = x - x.mean(-1, keepdim=True)
    rstd = (d.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    n = d * rstd
    w = s["weight"].view(G, -1)
    a = (n * w).flatten(-2) + s["bias"]
    z = None if s["z"] is None else s["z"].float()
    u, du = _act(a if z is None else z, s["act"])
    y = (u if z is None else a * u).to(dt)
    if s["op"] == "norm_fwd":
        return y
    gy = s["gy"].float()
    gz = None if z is None else (gy * a * du).to(dt)
    ga = gy * (du if z is None else u)
    gbias = ga.sum((0, 1))
    gweight = (ga * n.flatten(-2)).sum((0, 1))
    gn = ga.unflatten(-1, (G, C // G)) * w
    gx = rstd * (gn - gn.mean(-1, keepdim=True) - n * (gn * n).mean(-1, keepdim=True))
    return y, gx.flatten(-2).to(dt), gz, gweight, gbias


# ---- what a pass cannot do without, and the definition in 64 bits ----


def work(case):
    n = case["B"] * case["T"] * case["C"]
    es, rows = (4 if case["dtype"] == "f32" else 2), 4 * case["B"] * case["C"]
    op = case["op"]
    if op == "scan_step":  # g, x, y and the fp32 state in and out
        return {"bytes": n * (3 * es + 8), "flops": 8 * n}
    if op == "scan_fwd":  # g, x, y; state_in, state_out
        return {"bytes": 3 * n * es + 2 * rows, "flops": 8 * n}
    if op == "scan_train":  # g, x, gy, y, gg, gx; state_in, state_out and their gradients
        return {"bytes": 6 * n * es + 4 * rows, "flops": 24 * n}
    io = 3 if case["gate"] else 2  # x, (z,) y
    if op == "norm_fwd":
        return {"bytes": io * n * es + 8 * case["C"], "flops": 12 * n}
    return {"bytes": (2 * io) * n * es + 16 * case["C"], "flops": 36 * n}  # and gy, gx, (gz); weight, bias, gradients


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    T = case["T"]
    if case["op"].startswith("scan"):
        g = s["g"].double()
        f, i = torch.sigmoid(g), torch.sigmoid(-g)
        if case["op"] == "scan_step":
            h = f * s["state"].double() + i * x
            return h, h
        h = torch.empty_like(x)
        last = s["state_in"].double()
        for t in range(T):
            last = f[:, t] * last + i[:, t] * x[:, t]
            h[:, t] = last
        if case["op"] == "scan_fwd":
            return h, last
        gg, gx = torch.empty_like(x), torch.empty_like(x)
        mu = s["gstate"].double()  # the gradient of h_t through the later tokens
        for t in range(T - 1, -1, -1):
            lam = s["gy"][:, t].double() + mu
            before = h[:, t - 1] if t else s["state_in"].double()
            gg[:, t] = lam * (before - x[:, t]) * f[:, t] * i[:, t]
            gx[:, t] = lam * i[:, t]
            mu = lam * f[:, t]
        return h, last, gg, gx, mu
    G = case["groups"]
    x.requires_grad_()
    weight, bias = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    z = None if s["z"] is None else s["z"].double().requires_grad_()
    parts = x.reshape(case["B"], T, G, -1)
    mean = parts.mean(3, keepdim=True)
    var = (parts * parts).mean(3, keepdim=True) - mean * mean
    a = ((parts - mean) / torch.sqrt(var + _EPS)).reshape(x.shape) * weight + bias
    v = a if z is None else z
    v = v if case["act"] == "none" else torch.sigmoid(v) * (v if case["act"] == "silu" else 1)
    y = v if z is None else a * v
    if case["op"] == "norm_fwd":
        return y.detach()
    wrt = [x, weight, bias] + ([] if z is None else [z])
    grads = torch.autograd.grad(y, wrt, s["gy"].double())
    return y.detach(), grads[0], grads[3] if z is not None else None, grads[1], grads[2]
