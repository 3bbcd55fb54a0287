"""The gated group norm (forward and backward) against the fp64 oracle, the oracle against torch's
double precision and central differences, and the run of a layer's mixing step: recurrence, then
normalised and gated read-out, forward and backward.

Tolerances, in units of eps = 2^-24 and of the oracle's magnitude scales.  A sum over a group of D
values takes at most D / 32 + 32 additions per lane and 13 across lanes: k = D / 32 + 45 roundings
of partial sums.  The mean is then within (k + 2) eps of the largest |x| and the variance within
(k + 4) eps, so n is within (k + 8) eps of sn = max|x| r + |n|.  A logistic carries 2|v| eps from its
rounded exponent and 8 eps more, an activation's value or slope at most (4|v| + 16) eps of its terms.
    outputs, gz      (k + 4 max|v| + 32) eps      (v: the activation's argument)
    gx               (4 k + 8 max|v| + 96) eps    (n, ga, and two more group sums)
    gweight, gbias   (rows + k + 4 max|v| + 64) eps (a sum over the rows, in any order)
bf16 results add half a step, finfo.eps / 2 of the value.
"""
import numpy as np
import pytest

import oracle
from parity_util import to_gpu

EPS = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}
FAKE = 0x10000  # a 16-byte aligned, never dereferenced address


def _wkv():
    import linear_attention_rnn_wkv_b200 as wkv
    return wkv


def _td(dtype):
    import torch
    return torch.float32 if dtype == "f32" else torch.bfloat16


def _case(rows, G, D, seed, dtype="f32", gate=True, params=True, offset=1.0):
    """x, z, weight, bias, gy (z, weight, bias None where absent); values exact in the I/O dtype."""
    import torch
    r = np.random.default_rng(seed)
    io = lambda a: torch.from_numpy(a.astype(np.float32)).to(_td(dtype)).float().numpy()
    scale, shift = np.exp(r.normal(0, 1, (G, 1))), r.normal(0, offset, (G, 1))
    x = io((r.normal(0, 1, (rows, G, D)) * scale + shift).reshape(rows, G * D))
    z = io(r.normal(0, 1.5, (rows, G * D))) if gate else None
    w = (1 + 0.3 * r.normal(0, 1, G * D)).astype(np.float32) if params else None
    b = (0.3 * r.normal(0, 1, G * D)).astype(np.float32) if params else None
    return x, z, w, b, io(r.normal(0, 1, (rows, G * D)))


def _close(got, ref, scale, tol, half_step, what):
    got = got.float().cpu().numpy().astype(np.float64) if hasattr(got, "cpu") else np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    over = np.abs(got - ref) - (tol * scale + half_step * np.abs(ref) * (1 + tol) + 1e-36)
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(got - ref) / np.maximum(scale, 1e-300)):.3e} of scale, tol {tol:.3e}"


def _check(dtype, x, z, w, b, gy, G, eps=1e-5, act="silu", **out):
    """Forward and backward on the GPU against the oracle; returns the GPU results."""
    wkv = _wkv()
    td = _td(dtype)
    up = lambda a, t=None: None if a is None else to_gpu(a, t)
    how = dict(groups=G, eps=eps, act=act)
    X, Z, W, Bs, GY = up(x, td), up(z, td), up(w), up(b), up(gy, td)
    y = wkv.group_norm_gated(X, Z, W, Bs, **how)
    gx, gz, gw, gb = wkv.group_norm_gated_backward(X, Z, W, Bs, GY, **how)
    eps = float(np.float32(eps))
    yr, ys = oracle.group_norm_gated(x, z, w, b, G, eps, act)
    gxr, gzr, gwr, gbr, (sx, sz, sw, sb) = oracle.group_norm_gated_backward(x, z, w, b, gy, G, eps, act)
    C = x.shape[-1]
    rows, k = x.size // C, C // G / 32 + 45
    v = float(np.max(np.abs(z))) if z is not None else float(np.max(ys))  # |a| is below y's scale
    _close(y, yr, ys, (k + 4 * v + 32) * EPS, HALF[dtype], "y")
    _close(gx, gxr, sx, (4 * k + 8 * v + 96) * EPS, HALF[dtype], "gx")
    if z is None:
        assert gz is None
    else:
        _close(gz, gzr, sz, (k + 4 * v + 32) * EPS, HALF[dtype], "gz")
    _close(gw, gwr, sw, (rows + k + 4 * v + 64) * EPS, 0, "gweight")
    _close(gb, gbr, sb, (rows + k + 4 * v + 64) * EPS, 0, "gbias")
    return y, gx, gz, gw, gb


# ---- the oracle ----

@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("G,D", [(1, 7), (3, 4), (5, 1)])
def test_oracle_is_torch_in_double_and_its_differences(G, D, gate, act):
    import torch
    x, z, w, b, gy = (None if a is None else a.astype(np.float64) for a in _case(3, G, D, 10 * G + D, gate=gate))
    y, s = oracle.group_norm_gated(x, z, w, b, G, 1e-3, act)
    t = lambda a: None if a is None else torch.from_numpy(a)
    n = torch.nn.functional.group_norm(t(x), G, t(w), t(b), 1e-3)  # [rows, C]: a row is a sample
    f = {"none": lambda v: v, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[act]
    assert np.allclose(y, (n * f(t(z)) if gate else f(n)).numpy(), rtol=1e-12, atol=1e-14)
    assert np.all(s >= np.abs(y) * (1 - 1e-12))
    gx, gz, gw, gb, scales = oracle.group_norm_gated_backward(x, z, w, b, gy, G, 1e-3, act)
    for a, g, sc in zip((x, z, w, b), (gx, gz, gw, gb), scales):
        if a is None:
            assert g is None
            continue
        assert np.all(sc >= np.abs(g) * (1 - 1e-12))
        for i in np.ndindex(a.shape):
            v, d = a[i], 1e-5
            a[i] = v + d
            up = float(np.sum(gy * oracle.group_norm_gated(x, z, w, b, G, 1e-3, act)[0]))
            a[i] = v - d
            dn = float(np.sum(gy * oracle.group_norm_gated(x, z, w, b, G, 1e-3, act)[0]))
            a[i] = v
            # a difference quotient's error is d^2 / 6 of the third derivative, which grows as r^3
            assert abs((up - dn) / (2 * d) - g[i]) <= 1e-6 * max(1.0, abs(sc[i]))


# ---- refusals (no GPU) ----

def test_validation_without_launch():
    L = _wkv().lib()

    def fwd(rows=4, C=64, G=2, io=0, eps=1e-5, act=1, x=FAKE, z=None, w=None, b=None, y=FAKE):
        return L.group_norm_gated(rows, C, G, io, eps, act, x, z, w, b, y, None)

    def bwd(rows=4, C=64, G=2, io=0, eps=1e-5, act=1, x=FAKE, z=None, gy=FAKE, gx=FAKE, gz=None, gw=None, gb=None,
            ws=None, n=0):
        return L.group_norm_gated_backward(rows, C, G, io, eps, act, x, z, None, None, gy, gx, gz, gw, gb, ws, n, None)

    for call in (fwd, bwd):
        assert call(rows=-1) == 1 and call(C=-4) == 1 and call(rows=1 << 40, C=1 << 40, G=1) == 1
        assert call(io=7) == 3 and call(act=3) == 3
        assert call(G=0) == 1 and call(G=3) == 1 and call(G=-2) == 1
        assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
        assert call(C=1 << 32, G=1) == 3
        assert call(x=None) == 1 and call(x=FAKE + 8) == 2
        assert call(C=0, G=1) == 0
    assert fwd(rows=0, x=None, y=None) == 0
    assert fwd(y=None) == 1 and fwd(y=FAKE + 4) == 2 and fwd(z=FAKE + 4) == 2 and fwd(w=FAKE + 4) == 2
    assert bwd(gx=None) == 1 and bwd(gy=None) == 1 and bwd(z=FAKE) == 1 and bwd(gz=FAKE) == 1
    assert bwd(z=FAKE, gz=FAKE + 4) == 2 and bwd(gw=FAKE + 4, ws=FAKE, n=1 << 30) == 2
    need = L.group_norm_gated_backward_workspace_size(4, 64, 2, 0)
    assert need > 0 and need % (2 * 64 * 4) == 0
    assert bwd(gw=FAKE, ws=None) == 1 and bwd(gb=FAKE, ws=FAKE, n=need - 1) == 1
    assert bwd(rows=0) == 0
    assert L.group_norm_gated_backward_workspace_size(0, 64, 2, 0) == 0
    assert L.group_norm_gated_backward_workspace_size(4, 64, 3, 0) == 0
    assert L.group_norm_gated_backward_workspace_size(1 << 20, 4096, 64, 1) <= 8 * 4096 * 1184


def test_workspace_size_bound():
    """8 bytes per channel and block of rows, at most 1480 blocks (ten of 128 threads on each SM)."""
    size = _wkv().lib().group_norm_gated_backward_workspace_size
    most = 0
    for io in (0, 1):
        for D in (1, 3, 4, 8, 64, 65, 130, 520, 1030, 2048, 4096, 20000):
            for G in (1, 5, 64):
                for rows in (1, 7, 1000, 10 ** 7):
                    blocks, rest = divmod(size(rows, G * D, G, io), 8 * G * D)
                    assert rest == 0 and 1 <= blocks <= min(rows, 1480)
                    most = max(most, blocks)
    assert most == 1480
    assert size(0, 64, 1, 0) == size(8, 0, 1, 0) == size(8, 64, 3, 0) == size(8, 64, 0, 0) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    wkv = _wkv()
    t = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        wkv.group_norm_gated(t)
    with pytest.raises(TypeError):
        wkv.group_norm_gated_backward(t, None, None, None, t)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import torch
    wkv = _wkv()
    x = torch.zeros(2, 4, 6, device="cuda")
    p = torch.zeros(6, device="cuda")
    for bad in (dict(groups=4), dict(groups=0), dict(act="gelu"), dict(weight=p[:3]), dict(z=x[:1])):
        with pytest.raises(ValueError):
            wkv.group_norm_gated(x, **bad)
    for bad in (dict(z=x.bfloat16()), dict(weight=p.bfloat16()), dict(bias=p.cpu())):
        with pytest.raises(TypeError):
            wkv.group_norm_gated(x, **bad)
    with pytest.raises(TypeError):
        wkv.group_norm_gated(x.half())
    with pytest.raises(ValueError):
        wkv.group_norm_gated(x.transpose(0, 1))
    with pytest.raises(wkv.WkvError):
        wkv.group_norm_gated(x, eps=-1.0)
    with pytest.raises(ValueError):
        wkv.group_norm_gated_backward(x, None, None, None, x, gz=x.clone())
    with pytest.raises(ValueError):
        wkv.group_norm_gated_backward(x, x, None, None, x[:1])


# ---- the kernels ----

# (rows, groups, D): teams of 4, 8, 16, 32 lanes with 1, 2, 4 vectors, whole and part-filled, in
# 16-byte vectors, pairs and single channels; a block per group beyond; odd everything
SHAPES = [(1, 1, 1), (3, 2, 1), (5, 3, 2), (2, 5, 3), (7, 1, 4), (9, 4, 8), (4, 7, 16), (6, 3, 20), (3, 12, 64), (130, 5, 64),
          (2, 33, 64), (5, 3, 65), (3, 2, 100), (17, 2, 128), (3, 3, 250), (2, 2, 256), (3, 1, 500), (2, 1, 768),
          (3, 2, 1000), (2, 2, 1023), (3, 1, 1025), (2, 1, 4096), (1, 2, 5000), (3, 1, 4099)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(shape, dtype):
    rows, G, D = shape
    seed = 500 + rows * 131 + G * 17 + D
    _check(dtype, *_case(rows, G, D, seed, dtype), G)
    _check(dtype, *_case(rows, G, D, seed + 1, dtype, gate=False), G)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("params", [True, False])
def test_activations_and_missing_parameters(act, gate, params):
    for G, D in ((3, 64), (2, 27), (1, 700)):
        _check("f32", *_case(6, G, D, 600 + D, gate=gate, params=params), G, act=act, eps=64e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,G,D", [(5000, 12, 64), (2500, 1, 768), (3000, 5, 65), (700, 2, 2000), (1300, 1, 4100)])
def test_many_rows(rows, G, D, dtype):
    """More rows than one pass of the grid: the loops over rows and the sums over blocks."""
    _check(dtype, *_case(rows, G, D, 610 + D, dtype), G)


@pytest.mark.gpu
def test_flat_and_offset_groups():
    """A group of equal values (var = 0) gives n = 0 and gx finite; values far from zero keep the
    accuracy their own rounding leaves (the scale's max|x| r)."""
    x, z, w, b, gy = _case(8, 4, 64, 620, offset=100.0)
    x[0, :64] = 3.25
    x[1, 64:128] = 0.0
    y = _check("f32", x, z, w, b, gy, 4)[0].cpu().numpy()
    silu = z / (1 + np.exp(-z.astype(np.float64)))
    assert np.allclose(y[0, :64], b[:64] * silu[0, :64], rtol=1e-5, atol=1e-6)
    assert np.allclose(y[1, 64:128], b[64:128] * silu[1, 64:128], rtol=1e-5, atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 65, 700])
def test_non_finite_values_stay_in_their_group(D):
    wkv = _wkv()
    x, z, w, b, gy = _case(5, 3, D, 630)
    ref = wkv.group_norm_gated(to_gpu(x), to_gpu(z), to_gpu(w), to_gpu(b), groups=3).cpu().numpy()
    x[2, D + 5] = np.nan
    x[4, 3] = np.inf
    y = wkv.group_norm_gated(to_gpu(x), to_gpu(z), to_gpu(w), to_gpu(b), groups=3).cpu().numpy()
    bad = np.zeros(x.shape, bool)
    bad[2, D:2 * D] = bad[4, :D] = True
    assert np.array_equal(y[~bad], ref[~bad]) and not np.isfinite(y[bad]).any()


@pytest.mark.gpu
def test_empty_calls():
    import torch
    wkv = _wkv()
    e = torch.empty(0, 12, device="cuda")
    assert wkv.group_norm_gated(e, groups=3).shape == (0, 12)
    gx, gz, gw, gb = wkv.group_norm_gated_backward(e, e, None, None, e, groups=3)
    assert gx.shape == gz.shape == (0, 12) and not gw.any() and not gb.any()
    z = torch.empty(3, 0, device="cuda")
    assert wkv.group_norm_gated(z).shape == (3, 0)
    assert wkv.group_norm_gated_backward(z, None, None, None, z)[2].shape == (0,)


PAD, CANARY = 64, 12288.0


def _padded(shape, dtype):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * PAD,), float("nan"), dtype=dtype, device="cuda")
    buf[:PAD] = buf[-PAD:] = CANARY
    return buf, buf[PAD:PAD + n].view(*shape)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,G,D", [(5, 3, 64), (6, 2, 65), (3, 5, 12), (3, 1, 1030)])
def test_writes_exactly_its_outputs(rows, G, D, dtype):
    import torch
    wkv = _wkv()
    td = _td(dtype)
    x, z, w, b, gy = _case(rows, G, D, 640, dtype)
    C = G * D
    need = wkv.lib().group_norm_gated_backward_workspace_size(rows, C, G, 0 if dtype == "f32" else 1)
    bufs = {n: _padded(s, d) for n, s, d in (("y", (rows, C), td), ("gx", (rows, C), td), ("gz", (rows, C), td),
                                             ("ws", (need // 4,), torch.float32))}
    o = {n: v for n, (_, v) in bufs.items()}
    args = (to_gpu(x, td), to_gpu(z, td), to_gpu(w), to_gpu(b))
    wkv.group_norm_gated(*args, groups=G, y=o["y"])
    wkv.group_norm_gated_backward(*args, to_gpu(gy, td), groups=G, gx=o["gx"], gz=o["gz"], workspace=o["ws"])
    torch.cuda.synchronize()
    for n, (buf, v) in bufs.items():
        assert bool((buf[:PAD] == CANARY).all()) and bool((buf[-PAD:] == CANARY).all()), f"{n}: wrote outside"
        assert bool(torch.isfinite(v).all()), f"{n}: left unwritten"


@pytest.mark.gpu
def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph():
    import torch
    wkv = _wkv()
    x, z, w, b, gy = (to_gpu(a) for a in _case(3000, 6, 64, 650))

    def step():
        return (wkv.group_norm_gated(x, z, w, b, groups=6),) + wkv.group_norm_gated_backward(x, z, w, b, gy, groups=6)

    ref = step()
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs.append(step())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        for t in captured:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, ref))
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, ref))


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows equal a call on them alone, bit for bit (a row's values do
    not depend on the others)."""
    import torch
    wkv = _wkv()
    rows, C, last = 530000, 4096, 40
    assert rows * C > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(655)
    r = lambda: torch.empty(rows, C, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    x, z, gy = r(), r(), r()
    for groups in (64, 1):
        y = wkv.group_norm_gated(x, z, groups=groups)
        gx, gz, _, _ = wkv.group_norm_gated_backward(x, z, None, None, gy, groups=groups, want_params=False)
        tail = [t[-last:].contiguous() for t in (x, z, gy)]
        assert torch.equal(y[-last:], wkv.group_norm_gated(tail[0], tail[1], groups=groups))
        gx2, gz2, _, _ = wkv.group_norm_gated_backward(tail[0], tail[1], None, None, tail[2], groups=groups,
                                                       want_params=False)
        assert torch.equal(gx[-last:], gx2) and torch.equal(gz[-last:], gz2)


# ---- a layer's mixing step ----

@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_recurrence_then_read_out_forward_and_backward(graph):
    """y = group_norm(h) silu(z), h the gated recurrence from a stored state; the loss sum(gy y) +
    sum(gs state_out) differentiated through both calls' backwards, eagerly and as a replayed graph.
    The read-out's oracle takes the GPU's own h (each operator is held to its own tolerance), and the
    whole chain is checked against finite differences of the oracle's loss along random directions."""
    import torch
    wkv = _wkv()
    B, T, G, D = 2, 150, 3, 64
    C = G * D
    r = np.random.default_rng(660)
    f = lambda *s: r.normal(0, 1, s).astype(np.float32)
    g, x, s0, z, gy, gs = f(B, T, C) + 1, f(B, T, C), f(B, C), f(B, T, C), f(B, T, C), f(B, C)
    w, b = (1 + 0.1 * f(C)), 0.1 * f(C)
    dev = {n: to_gpu(a) for n, a in dict(g=g, x=x, s0=s0, z=z, gy=gy, gs=gs, w=w, b=b).items()}

    def step():
        h, so, carry = wkv.gated_scan_forward(dev["g"], dev["x"], state_in=dev["s0"], want_carry=True)
        y = wkv.group_norm_gated(h, dev["z"], dev["w"], dev["b"], groups=G)
        gh, gz, gw, gb = wkv.group_norm_gated_backward(h, dev["z"], dev["w"], dev["b"], dev["gy"], groups=G)
        return (h, so, y, gh, gz, gw, gb) + wkv.gated_scan_backward(dev["g"], dev["x"], carry, gh, gstate_out=dev["gs"])

    out = step()
    if graph:
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            out = step()
        for t in out:
            t.fill_(float("nan"))
        cg.replay()
    torch.cuda.synchronize()
    h, so, y, gh, gz, gw, gb, gg, gx, gs0 = (t.cpu().numpy().astype(np.float64) for t in out)
    eps = float(np.float32(1e-5))

    def loss(g, x, s0, z, w, b):
        h, _, so, _ = oracle.gated_scan(g, x, s0)
        return float(np.sum(gy * oracle.group_norm_gated(h, z, w, b, G, eps, "silu")[0]) + np.sum(gs * so))

    yr, ys = oracle.group_norm_gated(h, z, w, b, G, eps, "silu")
    _close(y, yr, ys, (D / 32 + 45 + 4 * np.max(np.abs(z)) + 32) * EPS, 0, "y")
    args = [a.astype(np.float64) for a in (g, x, s0, z, w, b)]
    for i, grad in enumerate((gg, gx, gs0, gz, gw, gb)):
        d = np.random.default_rng(670 + i).normal(0, 1, grad.shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        slope = (loss(*up) - loss(*dn)) / 2e-5
        # fp32 gradients of a few hundred terms each, against the sum's own magnitude
        assert abs(slope - float(np.sum(grad * d))) <= 2e-4 * float(np.sqrt(np.sum((grad * d) ** 2))) + 1e-4


@pytest.mark.gpu
def test_tokens_continue_a_prefill_through_the_read_out():
    """Serving: prefill and read-out, then one-token steps and read-outs of [N, L, C] rows."""
    import torch
    wkv = _wkv()
    B, T, G, D = 3, 40, 2, 64
    C = G * D
    r = np.random.default_rng(680)
    f = lambda *s: r.normal(0, 1, s).astype(np.float32)
    g, x, z = f(B, T, C) + 1, f(B, T, C), f(B, T, C)
    cut = T - 3
    G_, X, Z = to_gpu(g), to_gpu(x), to_gpu(z)
    h, state, _ = wkv.gated_scan_forward(G_[:, :cut].contiguous(), X[:, :cut].contiguous())
    ys = [wkv.group_norm_gated(h, Z[:, :cut].contiguous(), groups=G, act="sigmoid")]
    for t in range(cut, T):
        tok = wkv.gated_scan_step(G_[:, t:t + 1].contiguous(), X[:, t:t + 1].contiguous(), state.view(B, 1, C))
        ys.append(wkv.group_norm_gated(tok, Z[:, t:t + 1].contiguous(), groups=G, act="sigmoid"))
    hr, hs, _, _ = oracle.gated_scan(g, x)
    yr, ysc = oracle.group_norm_gated(hr, z, None, None, G, float(np.float32(1e-5)), "sigmoid")
    # an error e of h (relative to its scale) moves n by at most 3 e r max(scale): below 3 e times
    # y's scale where the state's scale is near its value; 1e-4 covers (4 T + 60) eps with a factor 8
    _close(torch.cat(ys, 1), yr, ysc, 1e-4, 0, "y")


@pytest.mark.gpu
def test_eagle_read_out():
    """The read-out of an Eagle prefill: 64-channel heads, RWKV-5's epsilon, SiLU gate."""
    import synth
    wkv = _wkv()
    spec = synth.eagle_spec_like("eagle_8x1024x768", 2, 70, 192, seed=690)
    w, r, k, v = (to_gpu(a) for a in synth.eagle_inputs(spec))
    y, _ = wkv.eagle_forward(w, r, k, v)
    rng = np.random.default_rng(691)
    f = lambda *s: rng.normal(0, 1, s).astype(np.float32)
    z, wt, b, gy = f(2, 70, 192), 1 + 0.1 * f(192), 0.1 * f(192), f(2, 70, 192)
    _check("f32", y.cpu().numpy(), z, wt, b, gy, 3, eps=64e-5)
