"""How accurate the gated linear recurrence stays over long memories: errors against the fp64
recurrence, with bounds that follow the recurrence itself instead of its length.

With f = sigma(g), i = 1 - f, s_t = f_t s_{t-1} + i_t |x_t| the state's magnitude scale and
eps = 2^-24, an error E of the state decays as the state does, so every step adds its own share:

    E_t = f_t E_{t-1} + eps (k_t (L_t f_t s_{t-1} + i_t |x_t|) + r s_t),   L_t = min(1, -log2 f_t)

  r    roundings of the carried state per step.  The long axis is split into spans of at least 16
       steps and the state is rounded once as it passes one: r = 1/16.  A sequence of at most 256
       steps may be walked token by token, two roundings each: r = 2.
  k_t  relative error of what a span does to a state, in units of eps: 2 |g| + 8 for the gate's
       smaller part (its exponent, exponential, 1 + e, reciprocal, product), at most 2 per step and 32
       steps for the share D = 1 - prod f of the state that the span replaces (or for prod f where that
       is at most 1/2), 34 for the state it builds from zero, and 4 per summary for the 16 summaries
       of a block: k_t = 2 |g| + 170.  It weighs i_t (s_{t-1} + |x_t|) where the step holds its
       state; i <= L f for i <= 1/2 by the concavity of -f log2 f.  A span that keeps at most half has
       the relative error of prod f, hence k_t prod f s: its L add up to 1 at least, and every
       f_t s_{t-1} times the decay after it is no less than prod f s.
An output adds 48 eps s_t: its own span's product (32), the state entering it, its sum.

The adjoint lam_t = gy_t + m_t, m_{t-1} = f_t lam_t is split alike, its scale p_t that of |gy|; a step of
the span's own part rounds twice, 2 * 32 + 64 + 2 = 130 per gy, and twice again in the span's walk:

    F_{t-1} = f_t F_t + eps (k_t L_t f_t p_t + 130 f_t |gy_t| + r p_t),   lam_t within F_t + 112 eps p_t
    gx = i lam                    within  i (lam's error + (2 |g| + 12) eps p)
    gg = f i (h_{t-1} - x) lam    within  f i (E_{t-1} + 36 eps (s + |x|)) p + f i (s + |x|) (lam's error
                                          + (4 |g| + 24) eps p),  s the scale of h_{t-1}
Second-order terms are below a thousandth of these: bounds are taken 1.01 times.  bf16 results add half a
step, finfo.eps / 2 of the value.
"""
import numpy as np
import pytest

from parity_util import to_gpu

EPS = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _exact(g, x, s0, gy, gs):
    """Outputs in fp64 and their bounds (before the output's own rounding): dicts by name."""
    g, x, s0, gy, gs = (np.asarray(a, np.float64) for a in (g, x, s0, gy, gs))
    B, T, C = g.shape
    rate = 2.0 if T <= 256 else 1 / 16
    f, i = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    k, L = 2 * np.abs(g) + 170, np.minimum(1, np.log2(1 + np.exp(-g)))
    h, s, E = (np.empty((B, T + 1, C)) for _ in range(3))
    h[:, 0], s[:, 0], E[:, 0] = s0, np.abs(s0), 0
    for t in range(T):
        h[:, t + 1] = f[:, t] * h[:, t] + i[:, t] * x[:, t]
        s[:, t + 1] = f[:, t] * s[:, t] + i[:, t] * np.abs(x[:, t])
        E[:, t + 1] = f[:, t] * E[:, t] + EPS * (k[:, t] * (L[:, t] * f[:, t] * s[:, t] + i[:, t] * np.abs(x[:, t])) +
                                                 rate * s[:, t + 1])
    gg, gx, bgg, bgx = (np.empty((B, T, C)) for _ in range(4))
    m, p, F = gs, np.abs(gs), np.zeros((B, C))
    for t in range(T - 1, -1, -1):
        ft, it, gt, xa = f[:, t], i[:, t], np.abs(g[:, t]), np.abs(x[:, t])
        lam, p = gy[:, t] + m, np.abs(gy[:, t]) + p
        err = F + 112 * EPS * p
        d, ds = h[:, t] - x[:, t], s[:, t] + xa
        gx[:, t], gg[:, t] = it * lam, ft * it * d * lam
        bgx[:, t] = it * (err + (2 * gt + 12) * EPS * p)
        bgg[:, t] = ft * it * ((E[:, t] + 36 * EPS * ds) * p + ds * (err + (4 * gt + 24) * EPS * p))
        F = ft * F + EPS * (k[:, t] * L[:, t] * ft * p + 130 * ft * np.abs(gy[:, t]) + rate * p)
        m, p = ft * lam, ft * p
    out = E + 48 * EPS * s
    val = dict(y=h[:, 1:], state_out=h[:, -1], carry=h[:, :-1:64], gg=gg, gx=gx, gstate_in=m)
    bound = dict(y=out[:, 1:], state_out=out[:, -1], carry=out[:, :-1:64], gg=bgg, gx=bgx,
                 gstate_in=F + 112 * EPS * p)
    return val, bound


def _check(got, val, bound, dtype="f32"):
    for name, a in got.items():
        a = a.float().cpu().numpy() if hasattr(a, "cpu") else a
        half = HALF[dtype] if name in ("y", "gg", "gx") else 0.0
        err, most = np.abs(a.astype(np.float64) - val[name]), 1.01 * bound[name] + half * np.abs(val[name]) * 1.01 + 1e-36
        worst = np.unravel_index(np.argmax(err / most), err.shape)
        assert np.all(np.isfinite(a)) and np.all(err <= most), \
            f"{name}{worst}: {a[worst]!r}, exactly {val[name][worst]!r}, off by {err[worst] / most[worst]:.2f} of the bound"


def _held(B, T, C):
    """One gate logit, input and gradient per channel for all steps: memories of 8 thousand to 24
    million steps, whose roundings, alike at every step, do not average out."""
    c = np.arange(B * C).reshape(B, 1, C)
    pick = lambda values, every: np.asarray(values, np.float32)[c // every % len(values)]
    g = pick([15.75, 16.25, 9.0, 12.0, 15.0, 17.0], 1)
    x = pick([0.6875, 0.0, -1.25], 6)
    full = lambda a: np.broadcast_to(a, (B, T, C)).copy()
    return full(g), full(x), pick([3.0, 0.375], 3)[:, 0], full(pick([0.3125, -0.75, 0.0], 2)), pick([2.0, -5.0], 5)[:, 0]


def _random(B, T, C, mean, std, seed, dtype="f32"):
    import torch
    r = np.random.default_rng(seed)
    io = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16).float().numpy()
    n = lambda *s: r.normal(0, 1, s)
    return io(mean + std * n(B, T, C)), io(n(B, T, C)), n(B, C).astype(np.float32), io(n(B, T, C)), n(B, C).astype(np.float32)


# ---- the bounds tell the forms apart (no GPU) ----

def _fma(a, b, c):
    return (a.astype(np.float64) * b + c).astype(np.float32)


def _states(kind, g, x, s0, span=16):
    """The states after each step in fp32: `naive` f h + i x per step; `products` spans of prod f and their
    own state; `complement` spans of 1 - prod f where that is below 1/2."""
    f, i = (1 / (1 + np.exp(-g.astype(np.float64)))).astype(np.float32), (1 / (1 + np.exp(g.astype(np.float64)))).astype(np.float32)
    B, T, C = g.shape
    out, h = np.empty_like(x), s0.copy()
    for t in range(T):
        ft, it, xt = f[:, t], i[:, t], x[:, t]
        if kind == "naive":
            h = _fma(ft, h, it * xt)
            out[:, t] = h
            continue
        if t % span == 0:
            start, A, D, H = h, np.ones_like(s0), np.zeros_like(s0), np.zeros_like(s0)
        holds = g[:, t] >= 0
        D = _fma(it, A, D)
        A = np.where(holds, _fma(-it, A, A), ft * A)
        H = np.where(holds, _fma(-it, H - xt, H), _fma(ft, H - xt, xt))
        if kind == "products":
            h = _fma(A, start, H)
        else:
            h = np.where(A > 0.5, start + _fma(-D, start, H), _fma(A, start, H))
        out[:, t] = h
    return out


@pytest.mark.parametrize("kind,passes", [("naive", False), ("products", False), ("complement", True)])
def test_bound_separates_the_forms(kind, passes):
    """f h + i x in fp32 and spans that keep only prod f drift over steady gates, to 17 and 7 times the
    bound; spans that keep the complement stay within it."""
    case = _held(1, 16384, 18)
    val, bound = _exact(*case)
    y = _states(kind, *case[:3])
    if passes:
        _check(dict(y=y), val, bound)
    else:
        with pytest.raises(AssertionError):
            _check(dict(y=y), val, bound)


# ---- the kernels ----

def _run(dtype, case):
    import torch
    import linear_attention_rnn_wkv_b200 as wkv
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    g, x, s0, gy, gs = case
    G, X, GY = (to_gpu(a, td) for a in (g, x, gy))
    y, so, carry = wkv.gated_scan_forward(G, X, state_in=to_gpu(s0), want_carry=True)
    gg, gx, gsi = wkv.gated_scan_backward(G, X, carry, GY, gstate_out=to_gpu(gs))
    _check(dict(y=y, state_out=so, carry=carry, gg=gg, gx=gx, gstate_in=gsi), *_exact(*case), dtype)


# full clusters over many strides (rows by TMA and by copies), clusters and single blocks of many
# channels, pairs of channels, sequences walked whole
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16384, 64), (1, 16384, 33), (2, 5000, 768), (1, 4100, 4040), (40, 700, 768), (20, 1000, 999),
                                   (40, 200, 4096), (40, 60, 3800), (2, 50, 66)], ids=lambda s: "x".join(map(str, s)))
def test_steady_gates_do_not_drift(shape, dtype):
    _run(dtype, _held(*shape))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g_mean,g_std", [(0.0, 0.01), (9.0, 0.5), (-9.0, 0.5), (0.0, 12.0), (2.0, 1.5)])
@pytest.mark.parametrize("shape", [(2, 600, 70), (1, 4100, 36), (1, 3000, 257)], ids=lambda s: "x".join(map(str, s)))
def test_gate_ranges_within_the_recurrences_own_bound(shape, g_mean, g_std, dtype):
    """Half-open gates, gates that hold for thousands of tokens, gates that forget at once, both ends
    mixed, and gates that mostly remember."""
    _run(dtype, _random(*shape, g_mean, g_std, seed=700, dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", [((40, 15, 3800), "f32"), ((40, 32, 3800), "bf16"), ((40, 63, 3801), "f32"),
                                         ((40, 64, 3801), "bf16"), ((40, 48, 3800), "bf16")],
                         ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_longest_sequences_walked_from_shared_memory(shape, dtype):
    """The backward that keeps a warp's steps in shared memory, at the most steps of each of its forms."""
    _run(dtype, _random(*shape, 2.0, 1.5, seed=710, dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [4096, 4097])
def test_both_ends_of_a_sequence_beyond_32_bit_offsets(C):
    """More than 2^31 elements: the last 256 tokens, from the state saved before them, and the first 256, whose
    adjoint a closed gate at the 257th cuts off from the rest, against the fp64 recurrence element by element."""
    import torch
    import linear_attention_rnn_wkv_b200 as wkv
    T, n = 64 * 8300, 256
    assert T * C > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(720)
    r = lambda: torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g, x, gy = r(), r(), r()
    g[:, n] = -torch.inf
    y, so, carry = wkv.gated_scan_forward(g, x, want_carry=True)
    gg, gx, gsi = wkv.gated_scan_backward(g, x, carry, gy)
    assert not gg[:, n].any() and torch.equal(y[:, n], x[:, n])
    zeros = np.zeros((1, C), np.float32)
    up = lambda *a: [t.float().cpu().numpy() for t in a]
    for at, s0, ends in ((0, zeros, dict(gstate_in=gsi)), (T - n, up(carry[:, (T - n) // 64])[0], dict(state_out=so))):
        span = slice(at, at + n)
        case = up(g[:, span], x[:, span], gy[:, span])
        val, bound = _exact(case[0], case[1], s0, case[2], zeros)
        _check(dict(y=y[:, span], gg=gg[:, span], gx=gx[:, span], carry=carry[:, at // 64:at // 64 + n // 64], **ends),
               val, bound, "bf16")
