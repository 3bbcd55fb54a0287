"""The gated linear recurrence h_t = f_t h_{t-1} + (1 - f_t) x_t, f = sigma(g): forward, backward
and one-token step against the fp64 oracle, and the oracle against the unrolled sum and central
differences.

Tolerances, in units of eps = 2^-24 and of each value's magnitude scale (the oracle's recurrence
on absolute values).  A gate's smaller part carries 2|g| eps from the rounded exponent (g log2 e
and the constant), 4 eps from the exponential (2^-22), 4 eps from 1 + e, its reciprocal and the
product: below (2|g| + 8) eps; it enters a state with weight at most 2 of the state's scale.  A
step rounds its difference and its sum, 2 eps; the state entering a warp's steps comes from
summaries whose factors round once per step and once per fold, below another 2 eps per step in
all.  So
    states, outputs       (4 T + 4 max|g| + 40) eps
and a gate's gradient, the product of a state, an adjoint and f (1 - f), twice that plus its own
factors', a further 6 max|g| eps.  bf16 results add half a step, finfo.eps / 2 of the value.
"""
import ctypes

import numpy as np
import pytest
from hypothesis import given, settings, strategies as st

import oracle
from parity_util import to_gpu

EPS = 2.0 ** -24
FAKE = 0x10000  # a 16-byte aligned, never dereferenced address


def _wkv():
    import linear_attention_rnn_wkv_b200 as wkv
    return wkv


def _case(B, T, C, seed, dtype="f32", g_mean=2.0, g_std=1.5):
    """g, x, state_in, gy, gstate; values exact in the I/O dtype."""
    r = np.random.default_rng(seed)
    import torch
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    f = lambda *s, mean=0.0, std=1.0: (mean + std * r.normal(0, 1, s)).astype(np.float32)
    io = lambda a: torch.from_numpy(a).to(td).float().numpy()
    return (io(f(B, T, C, mean=g_mean, std=g_std)), io(f(B, T, C)), f(B, C), io(f(B, T, C)), f(B, C))


def _tol(T, g):
    gm = float(np.max(np.abs(g[np.isfinite(g)]), initial=0.0))
    return (4 * T + 4 * gm + 40) * EPS


def _assert_close(got, ref, scale, tol, half_step, what):
    got = got.float().cpu().numpy().astype(np.float64) if hasattr(got, "cpu") else np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    over = np.abs(got - ref) - (tol * scale + half_step * np.abs(ref) * (1 + tol) + 1e-36)
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(got - ref) / np.maximum(scale, 1e-300)):.3e} of scale, tol {tol:.3e}"


def _td(dtype):
    import torch
    return torch.float32 if dtype == "f32" else torch.bfloat16


HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _check_train(dtype, g, x, s0, gy, gs, use_state=True):
    """Forward with carry and backward on the GPU against the oracle; returns the GPU results."""
    wkv = _wkv()
    td = _td(dtype)
    G, X, GY = to_gpu(g, td), to_gpu(x, td), to_gpu(gy, td)
    S0, GS = (to_gpu(s0), to_gpu(gs)) if use_state else (None, None)
    y, so, carry = wkv.gated_scan_forward(G, X, state_in=S0, want_carry=True)
    gg, gx, gsi = wkv.gated_scan_backward(G, X, carry, GY, gstate_out=GS)
    s0, gs = (s0, gs) if use_state else (None, None)
    yr, sr, sor, ssr = oracle.gated_scan(g, x, s0)
    ggr, gxr, gsr, (sg, sx, ss) = oracle.gated_scan_backward(g, x, gy, s0, gs)
    T, tol = g.shape[1], _tol(g.shape[1], g)
    _assert_close(y, yr, sr, tol, HALF[dtype], "y")
    _assert_close(so, sor, ssr, tol, 0, "state_out")
    _assert_close(gx, gxr, sx, 2 * tol, HALF[dtype], "gx")
    _assert_close(gg, ggr, sg, 2 * tol + 6 * float(np.max(np.abs(g[np.isfinite(g)]), initial=0)) * EPS, HALF[dtype], "gg")
    _assert_close(gsi, gsr, ss, tol, 0, "gstate_in")
    for j in range(carry.shape[1]):
        ref, sc = (s0, np.abs(s0)) if j == 0 and s0 is not None else (np.zeros(so.shape), np.zeros(so.shape)) \
            if j == 0 else (yr[:, 64 * j - 1], sr[:, 64 * j - 1])
        _assert_close(carry[:, j], ref, sc, tol, 0, f"carry {j}")
    return y, so, carry, gg, gx, gsi


# ---- the oracle ----

SETTINGS = settings(max_examples=40, deadline=None, derandomize=True)


@SETTINGS
@given(B=st.integers(1, 2), T=st.integers(1, 20), C=st.integers(1, 4), given_state=st.booleans(),
       g_std=st.floats(0.1, 6.0), seed=st.integers(0, 2**31 - 1))
def test_oracle_recurrence_is_the_unrolled_sum(B, T, C, given_state, g_std, seed):
    """h_t = sum_{j<=t} (prod_{j<k<=t} f_k) (1 - f_j) x_j + (prod_{k<=t} f_k) h_{-1}, a convex
    combination of the x_j and the state; the scale bounds it."""
    r = np.random.default_rng(seed)
    g, x = r.normal(0, g_std, (B, T, C)), r.normal(0, 1, (B, T, C))
    s0 = r.normal(0, 1, (B, C)) if given_state else None
    y, s, so, ss = oracle.gated_scan(g, x, s0)
    f = 1 / (1 + np.exp(-g))
    for t in range(T):
        tot = np.prod(f[:, :t + 1], axis=1) * (0 if s0 is None else s0)
        for j in range(t + 1):
            tot = tot + np.prod(f[:, j + 1:t + 1], axis=1) / (1 + np.exp(g[:, j])) * x[:, j]
        assert np.allclose(y[:, t], tot, rtol=1e-12, atol=1e-13)
    assert np.array_equal(so, y[:, -1]) and np.array_equal(ss, s[:, -1])
    assert np.all(s >= np.abs(y) * (1 - 1e-12))


@SETTINGS
@given(B=st.integers(1, 2), T=st.integers(1, 6), C=st.integers(1, 2), seed=st.integers(0, 2**31 - 1))
def test_oracle_backward_against_central_differences(B, T, C, seed):
    r = np.random.default_rng(seed)
    g, x, gy = (r.normal(0, 1.5, (B, T, C)) for _ in range(3))
    s0, gs = r.normal(0, 1, (B, C)), r.normal(0, 1, (B, C))

    def loss():
        y, _, so, _ = oracle.gated_scan(g, x, s0)
        return float(np.sum(gy * y) + np.sum(gs * so))

    gg, gx, g0, (sg, sx, ss) = oracle.gated_scan_backward(g, x, gy, s0, gs)
    for a, grad, sc in ((g, gg, sg), (x, gx, sx), (s0, g0, ss)):
        assert np.all(sc >= np.abs(grad) * (1 - 1e-12))
        for i in np.ndindex(a.shape):
            v, d = a[i], 1e-5
            a[i] = v + d
            up = loss()
            a[i] = v - d
            dn = loss()
            a[i] = v
            assert abs((up - dn) / (2 * d) - grad[i]) <= 1e-7


# ---- refusals (no GPU) ----

def test_validation_without_launch():
    L = _wkv().lib()

    def fwd(B, T, C, io=0, g=FAKE, x=FAKE, s=None, y=FAKE, so=None, carry=None):
        return L.gated_scan_forward(B, T, C, io, g, x, s, y, so, carry, None)

    def bwd(B, T, C, io=0, g=FAKE, carry=FAKE, gs=None, gg=FAKE, gx=FAKE, gsi=None):
        return L.gated_scan_backward(B, T, C, io, g, FAKE, carry, FAKE, gs, gg, gx, gsi, None)

    for call in (fwd, bwd):
        assert call(-1, 4, 4) == 1                   # negative size
        assert call(1 << 40, 1 << 40, 4) == 1        # product overflows
        assert call(1, 4, 4, io=7) == 3              # unknown dtype
        assert call(1, 4, 4, g=None) == 1            # null input
        assert call(1, 4, 4, g=FAKE + 8) == 2        # misaligned input
        assert call(1 << 28, 1, 4) == 3              # more blocks than a launch holds
        assert call(1 << 23, 1, 1024) == 3
        assert call(1, 1, 1 << 23) == 3              # 32-bit offsets within a tile
        assert call(0, 4, 4) == 0 and call(3, 4, 0) == 0
    assert fwd(1, 4, 4, y=None) == 1
    assert fwd(1, 4, 4, y=FAKE + 4) == 2 and fwd(1, 4, 4, s=FAKE + 4) == 2
    assert fwd(1, 4, 4, so=FAKE + 4) == 2 and fwd(1, 4, 4, carry=FAKE + 4) == 2
    assert bwd(1, 4, 4, carry=None) == 1 and bwd(1, 4, 4, gg=None) == 1 and bwd(1, 4, 4, gx=None) == 1
    assert bwd(1, 4, 4, gsi=FAKE + 4) == 2 and bwd(1, 4, 4, gs=FAKE + 4) == 2
    assert bwd(2, 0, 4, carry=None, g=None, gg=None, gx=None) == 0  # nothing to write
    assert fwd(2, 0, 4, g=None, x=None, y=None) == 0

    step = lambda N, g=FAKE, st_=FAKE, y=FAKE, io=0: L.gated_scan_step(N, 2, 4, io, g, FAKE, st_, y, None)
    assert step(-1) == 1 and step(2, g=None) == 1 and step(2, st_=None) == 1 and step(2, y=FAKE + 4) == 2
    assert step(2, io=5) == 3 and step(0) == 0
    assert L.gated_scan_carry_size(2, 64, 5) == 2 * 1 * 5 * 4
    assert L.gated_scan_carry_size(2, 65, 5) == 2 * 2 * 5 * 4
    assert L.gated_scan_carry_size(2, 0, 5) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    wkv = _wkv()
    t = torch.zeros(1, 4, 4)
    for call in (lambda: wkv.gated_scan_forward(t, t), lambda: wkv.gated_scan_step(t, t, t),
                 lambda: wkv.gated_scan_backward(t, t, torch.zeros(1, 1, 4), t)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import torch
    wkv = _wkv()
    g = torch.zeros(2, 4, 6, device="cuda")
    carry = torch.zeros(2, 1, 6, device="cuda")
    with pytest.raises(TypeError):
        wkv.gated_scan_forward(g, g.bfloat16())
    with pytest.raises(TypeError):
        wkv.gated_scan_forward(g.half(), g.half())
    with pytest.raises(ValueError):
        wkv.gated_scan_forward(g, g[:1])
    with pytest.raises(ValueError):
        wkv.gated_scan_forward(g.transpose(0, 1), g.transpose(0, 1))
    with pytest.raises(ValueError):
        wkv.gated_scan_forward(g[0], g[0])
    with pytest.raises(ValueError):
        wkv.gated_scan_forward(g, g, state_in=torch.zeros(2, 5, device="cuda"))
    with pytest.raises(ValueError):
        wkv.gated_scan_backward(g, g, carry[:, :0], g)
    with pytest.raises(TypeError):
        wkv.gated_scan_backward(g, g, carry, g.bfloat16())
    with pytest.raises(TypeError):
        wkv.gated_scan_step(g, g, g.bfloat16())
    with pytest.raises(ValueError):
        wkv.gated_scan_step(g, g, g[:, :, :3])
    off = torch.zeros(49, device="cuda")[1:].view(2, 4, 6)  # contiguous, 4 bytes past a boundary
    with pytest.raises(wkv.WkvError):
        wkv.gated_scan_forward(off, g)


# ---- the kernels ----

# one token, one warp's steps and its neighbours, a tile and its neighbours, several tiles and
# strides of a cluster; widths below, at and above a warp's channels, odd and even
SHAPES = [(1, 1, 1), (2, 1, 64), (3, 7, 5), (1, 8, 33), (2, 9, 130), (1, 16, 257), (5, 17, 31), (2, 64, 64),
          (2, 65, 66), (1, 127, 32), (1, 128, 96), (2, 129, 34), (1, 255, 257), (1, 256, 64), (2, 300, 36),
          (1, 1000, 8), (1, 1024, 40), (1, 1025, 3), (3, 1100, 130), (1, 2049, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_training_step_matches_oracle(shape, dtype):
    _check_train(dtype, *_case(*shape, seed=100 + sum(shape), dtype=dtype))
    _check_train(dtype, *_case(*shape, seed=200 + sum(shape), dtype=dtype), use_state=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(40, 700, 768), (2, 700, 4096), (1, 3000, 1000), (1, 4100, 256), (1, 4300, 33),
                                   (1, 4100, 4040), (32, 4100, 196), (2, 1000, 488), (1, 4000, 760),
                                   (1, 4100, 257), (1, 3300, 769), (3, 1001, 257),
                                   (40, 3, 3800), (40, 13, 3800), (40, 27, 3800), (40, 60, 3800), (40, 64, 3800),
                                   (40, 130, 3800), (33, 50, 1199), (70, 1, 1000), (50, 3, 515), (30, 30, 1002), (20, 60, 999),
                                   (20, 40, 1000), (20, 64, 1000), (40, 56, 3800), (40, 45, 3801)],
                         ids=lambda s: "x".join(map(str, s)))
def test_training_step_configurations(shape, dtype):
    """Many channels (the time axis in one block, or few), few channels and a long axis (full clusters,
    each tile length and channels per lane), long sequences whose pairs of channels fill the device
    in clusters or in single blocks, rows that TMA cannot stage (the same splits), short sequences
    of every length class, of few and of many channels; ragged last tiles and channel groups throughout."""
    _check_train(dtype, *_case(*shape, seed=300 + sum(shape), dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("g_mean,g_std", [(0.0, 0.01), (9.0, 0.5), (-9.0, 0.5), (0.0, 12.0)])
def test_gate_ranges(g_mean, g_std):
    """Half-open gates, gates that hold for thousands of tokens, gates that forget at once, and
    both ends mixed."""
    _check_train("f32", *_case(2, 600, 70, seed=400, g_mean=g_mean, g_std=g_std))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_boundaries_and_padding(dtype):
    """g = -inf replaces the state exactly (whatever its size) and so does -200 (f underflows);
    g = +inf and 200 keep it: exactly within one warp's steps, and to its rounding from span to
    span (the state entering a span is formed from summaries, so its bits may differ from the
    output before it, but both are within tol of one exact value, hence 2 tol apart).  Gradients
    of infinite gates are zero."""
    g, x, s0, gy, gs = _case(2, 400, 36, seed=410, dtype=dtype)
    g[0, 150] = -np.inf
    g[1, 300:] = np.inf
    x[1, 300:] = 7.0
    g[0, 200] = -200.0
    g[0, 250] = 200.0
    s0 = s0 * 1e6
    y, so, _, gg, gx, _ = _check_train(dtype, g, x, s0, gy, gs)
    y, gg, gx = (a.float().cpu().numpy() for a in (y, gg, gx))
    assert np.array_equal(y[0, 150], x[0, 150]) and np.array_equal(y[0, 200], x[0, 200])
    apart = 2 * _tol(400, g) * np.max(np.abs(x)) + 2 * HALF[dtype] * np.abs(y)
    assert np.all(np.abs(y[0, 250] - y[0, 249]) <= apart[0, 249])
    assert np.array_equal(y[1, 300:304], np.broadcast_to(y[1, 300], y[1, 300:304].shape))
    assert np.all(np.abs(y[1, 300:] - y[1, 299]) <= apart[1, 299])
    assert np.all(np.abs(so.cpu().numpy()[1] - y[1, 299]) <= apart[1, 299])
    assert not gg[0, 150].any() and not gg[1, 300:].any() and not gx[1, 300:].any()


@pytest.mark.gpu
def test_non_finite_values_stay_in_their_channel():
    import torch
    wkv = _wkv()
    g, x, s0, gy, _ = _case(2, 300, 40, seed=420)
    ref = wkv.gated_scan_forward(to_gpu(g), to_gpu(x), state_in=to_gpu(s0))[0].cpu().numpy()
    g[0, 140, 3] = np.nan
    x[1, 20, 39] = np.inf
    s0[1, 0] = np.nan
    y, so, _ = wkv.gated_scan_forward(to_gpu(g), to_gpu(x), state_in=to_gpu(s0))
    y = y.cpu().numpy()
    bad = ~np.isfinite(y)
    expect = np.zeros_like(bad)
    expect[0, 140:, 3] = expect[1, 20:, 39] = expect[1, :, 0] = True
    assert np.array_equal(bad, expect)
    assert np.array_equal(y[~bad], ref[~bad])
    assert np.array_equal(~np.isfinite(so.cpu().numpy()), expect[:, -1])


@pytest.mark.gpu
def test_resume_and_step_continue_the_sequence():
    """Prefill [0, cut), [cut, T - 2) from its state, then two one-token steps."""
    import torch
    wkv = _wkv()
    B, T, C, cut = 3, 333, 50, 171
    for dtype in ("f32", "bf16"):
        g, x, s0, _, _ = _case(B, T, C, seed=430, dtype=dtype)
        G, X = to_gpu(g, _td(dtype)), to_gpu(x, _td(dtype))
        state = to_gpu(s0)
        ys = []
        for lo, hi in ((0, cut), (cut, T - 2)):
            y, _, _ = wkv.gated_scan_forward(G[:, lo:hi].contiguous(), X[:, lo:hi].contiguous(), state_in=state,
                                             state_out=state)  # in place
            ys.append(y)
        for t in (T - 2, T - 1):
            ys.append(wkv.gated_scan_step(G[:, t:t + 1].contiguous(), X[:, t:t + 1].contiguous(), state.view(B, 1, C)))
        yr, sr, sor, ssr = oracle.gated_scan(g, x, s0)
        _assert_close(torch.cat(ys, 1), yr, sr, _tol(T, g), HALF[dtype], "y")
        _assert_close(state, sor, ssr, _tol(T, g), 0, "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 2, 5), (2, 3, 64), (8, 12, 768), (7, 3, 1001)], ids=lambda s: "x".join(map(str, s)))
def test_step_matches_oracle(shape, dtype):
    wkv = _wkv()
    N, L, C = shape
    g, x, _, _, _ = _case(N, L, C, seed=440, dtype=dtype)
    s0 = np.random.default_rng(441).normal(0, 1, shape).astype(np.float32)
    state = to_gpu(s0)
    y = wkv.gated_scan_step(to_gpu(g, _td(dtype)), to_gpu(x, _td(dtype)), state)
    flat = lambda a: a.reshape(N * L, 1, C)
    yr, sr, _, _ = oracle.gated_scan(flat(g), flat(x), s0.reshape(N * L, C))
    _assert_close(y, yr.reshape(shape), sr.reshape(shape), _tol(1, g), HALF[dtype], "y")
    _assert_close(state, yr.reshape(shape), sr.reshape(shape), _tol(1, g), 0, "state")


@pytest.mark.gpu
def test_empty_sequence_passes_the_state_through():
    import torch
    wkv = _wkv()
    e = torch.empty(2, 0, 37, device="cuda")
    s = torch.randn(2, 37, device="cuda")
    y, so, carry = wkv.gated_scan_forward(e, e, state_in=s, want_carry=True)
    assert y.shape == e.shape and carry.shape == (2, 0, 37) and torch.equal(so, s)
    assert not wkv.gated_scan_forward(e, e)[1].any()
    assert torch.equal(wkv.gated_scan_backward(e, e, carry, e, gstate_out=s)[2], s)
    assert not wkv.gated_scan_backward(e, e, carry, e)[2].any()
    for shape in ((0, 5, 4), (2, 5, 0)):
        z = torch.empty(shape, device="cuda")
        y, so, carry = wkv.gated_scan_forward(z, z, want_carry=True)
        wkv.gated_scan_backward(z, z, carry, z)
        wkv.gated_scan_step(z, z, z.clone())


PAD, CANARY = 64, 12288.0  # elements each side (16-byte aligned); exact in fp32 and bf16


def _padded(shape, dtype):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * PAD,), float("nan"), dtype=dtype, device="cuda")
    buf[:PAD] = buf[-PAD:] = CANARY
    return buf, buf[PAD:PAD + n].view(*shape)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 77, 96), (1, 300, 65), (3, 5, 36), (1, 1030, 130)], ids=lambda s: "x".join(map(str, s)))
def test_writes_exactly_its_outputs(shape, dtype):
    import torch
    wkv = _wkv()
    B, T, C = shape
    td = _td(dtype)
    g, x, s0, gy, gs = _case(B, T, C, seed=450, dtype=dtype)
    G, X = to_gpu(g, td), to_gpu(x, td)
    bufs = {n: _padded(s, d) for n, s, d in (("y", shape, td), ("so", (B, C), torch.float32),
                                             ("carry", (B, (T + 63) // 64, C), torch.float32), ("gg", shape, td),
                                             ("gx", shape, td), ("gsi", (B, C), torch.float32))}
    o = {n: v for n, (_, v) in bufs.items()}
    wkv.gated_scan_forward(G, X, state_in=to_gpu(s0), y=o["y"], state_out=o["so"], carry=o["carry"])
    wkv.gated_scan_backward(G, X, o["carry"], to_gpu(gy, td), gstate_out=to_gpu(gs), gg=o["gg"], gx=o["gx"],
                            gstate_in=o["gsi"])
    torch.cuda.synchronize()
    for n, (buf, v) in bufs.items():
        assert bool((buf[:PAD] == CANARY).all()) and bool((buf[-PAD:] == CANARY).all()), f"{n}: wrote outside its output"
        assert bool(torch.isfinite(v).all()), f"{n}: left unwritten"


@pytest.mark.gpu
def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph():
    """Two streams at once and a replayed graph give the bits of a plain call."""
    import torch
    wkv = _wkv()
    g, x, s0, gy, gs = _case(2, 1500, 260, seed=460)
    G, X, S0, GY, GS = (to_gpu(a) for a in (g, x, s0, gy, gs))

    def step():
        y, so, carry = wkv.gated_scan_forward(G, X, state_in=S0, want_carry=True)
        return (y, so, carry) + wkv.gated_scan_backward(G, X, carry, GY, gstate_out=GS)

    ref = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
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
        for a, b in zip(captured, ref):
            assert torch.equal(a, b)
    for o in outs:
        for a, b in zip(o, ref):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [4096, 4097])
def test_offsets_beyond_32_bits(C):
    """More than 2^31 elements: the last tokens of a long sequence, forward and backward, equal a call
    on them alone from the state saved before them (to twice the last tokens' tolerance: two runs of
    the same recurrence from one state)."""
    import torch
    wkv = _wkv()
    T, last = 64 * 8300, 256
    assert T * C > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(470)
    r = lambda: torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g, x, gy = r(), r(), r()
    y, so, carry = wkv.gated_scan_forward(g, x, want_carry=True)
    gg, gx, _ = wkv.gated_scan_backward(g, x, carry, gy)
    tail = [t[:, -last:].contiguous() for t in (g, x, gy)]
    y2, so2, carry2 = wkv.gated_scan_forward(tail[0], tail[1], state_in=carry[:, (T - last) // 64].contiguous(),
                                             want_carry=True)
    gg2, gx2, _ = wkv.gated_scan_backward(tail[0], tail[1], carry2, tail[2])
    tol = 2 * _tol(last, tail[0].float().cpu().numpy())
    big = max(float(t.abs().max()) for t in (x, gy))  # bounds every state; the adjoint at most 1 / (1 - f) times gy
    reach = big / float(torch.sigmoid(-tail[0].float()).min())
    for a, b, scale in ((y[:, -last:], y2, big), (gx[:, -last:], gx2, big), (gg[:, -last:], gg2, 2 * big * reach)):
        a, b = a.float(), b.float()
        assert bool(((a - b).abs() <= 2 * tol * scale + 2 * HALF["bf16"] * b.abs()).all())
    assert bool(((so - so2).abs() <= tol * big).all())
    # and the first tokens, which the backward reaches last
    head = [t[:, :last].contiguous() for t in (g, x)]
    assert torch.equal(wkv.gated_scan_forward(*head)[0][:, :64], y[:, :64])
