"""fp64 oracle for the gated linear recurrence -- TEST INFRASTRUCTURE ONLY.

    a_t = exp(-decay softplus(a_param) sigmoid(a_gate_t)), or sigmoid(a_gate_t) without a_param
    h_t = a_t h_{t-1} + s_t x_t sigmoid(x_gate_t),  s_t = sqrt(1 - a_t^2), 1 - a_t or 1
    y_t = h_t act(z_t)

Plain numpy in float64, token by token.  With `magnitude`, every sum is taken over its terms'
absolute values, for an error bound.
"""
import numpy as np

from .layer_ops import _f64
from .scan_ops import sigmoid, softplus

GELU = 2 * np.sqrt(2 / np.pi)


def inner(act, z):
    """act(z) = z sigmoid(inner(z))."""
    return z if act == "silu" else GELU * (z + 0.044715 * z ** 3)


def slope(act, z, magnitude=False):
    """Derivative of act at z."""
    p, rest = sigmoid(inner(act, z)), sigmoid(-inner(act, z))
    d = 1.0 if act == "silu" else GELU * (1 + 3 * 0.044715 * z * z)
    second = z * p * rest * d
    return p + (np.abs(second) if magnitude else second)


def exponents(a_gate, a_param, decay):
    """-log a of every token and channel."""
    return softplus(-a_gate) if a_param is None else decay * softplus(a_param) * sigmoid(a_gate)


def scale_of(kind, w):
    return {"sqrt": lambda: np.sqrt(-np.expm1(-2 * w)), "linear": lambda: -np.expm1(-w), "one": lambda: np.ones_like(w)}[kind]()


def _terms(x, a_gate, a_param, x_gate, z, input_scale, decay, activation):
    x, a_gate, a_param, x_gate, z = map(_f64, (x, a_gate, a_param, x_gate, z))
    w = exponents(a_gate, a_param, decay)
    p = np.ones_like(x) if x_gate is None else sigmoid(x_gate)
    f = np.ones_like(x) if z is None else z * sigmoid(inner(activation, z))
    return x, a_gate, a_param, z, w, p, f, scale_of(input_scale, w)


def _walk(w, b, h0, cu):
    h, last = np.zeros(w.shape), np.array(h0)
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        for t in range(lo, hi):
            last[n] = h[t] = np.exp(-w[t]) * last[n] + b[t]
    return h, last


def linear_recurrence(x, a_gate, cu, a_param=None, x_gate=None, z=None, init_state=None, input_scale="sqrt", decay=8.0,
                      activation="silu", magnitude=False):
    """(y [T, C], final states [N, C]); rows that no sequence covers are NaN in y."""
    x, _, _, _, w, p, f, s = _terms(x, a_gate, a_param, x_gate, z, input_scale, decay, activation)
    h0 = np.zeros((len(cu) - 1, x.shape[1])) if init_state is None else _f64(init_state)
    if magnitude:
        x, h0, f = np.abs(x), np.abs(h0), np.abs(f)
    h, last = _walk(w, s * x * p, h0, cu)
    y = h * f
    y[cu[-1]:] = np.nan
    return y, last


def linear_recurrence_bwd(x, a_gate, cu, d_out, a_param=None, x_gate=None, z=None, init_state=None, d_final_state=None,
                          input_scale="sqrt", decay=8.0, activation="silu", magnitude=False):
    """dict of dx, da_gate, dx_gate, dz, da_param, d_init_state, those of absent inputs left out."""
    x, ag, ap, z, w, p, f, s = _terms(x, a_gate, a_param, x_gate, z, input_scale, decay, activation)
    T, C = x.shape
    N = len(cu) - 1
    h0 = np.zeros((N, C)) if init_state is None else _f64(init_state)
    gT = np.zeros((N, C)) if d_final_state is None else _f64(d_final_state)
    dy = _f64(d_out)
    if magnitude:
        x, h0, gT, dy, f = map(np.abs, (x, h0, gT, dy, f))
    v, a, m = x * p, np.exp(-w), -np.expm1(-w)
    h, _ = _walk(w, s * v, h0, cu)
    with np.errstate(divide="ignore", invalid="ignore"):
        ds = {"sqrt": lambda: np.where(m > 0, a * a / s, 0.0), "linear": lambda: a, "one": lambda: np.zeros_like(a)}[input_scale]()  # -ds/du
    if magnitude:
        ds = -ds
    G, old = np.zeros((T, C)), np.zeros((T, C))
    d_init = np.array(gT)
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        g = gT[n]
        for t in range(hi - 1, lo - 1, -1):
            G[t] = g + dy[t] * f[t]
            old[t] = h[t - 1] if t > lo else h0[n]
            g = a[t] * G[t]
        d_init[n] = g
    du = G * (a * old - v * ds)  # dL/d(-w)
    out = dict(dx=G * s * p, d_init_state=d_init)
    if x_gate is not None:
        out["dx_gate"] = G * s * v * sigmoid(-_f64(x_gate))
    if z is not None:
        out["dz"] = dy * h * (slope(activation, z, True) if magnitude else slope(activation, z))
    sign = 1.0 if magnitude else -1.0
    if ap is None:
        out["da_gate"] = du * m
    else:
        out["da_gate"] = sign * du * w * sigmoid(-ag)
        out["da_param"] = sign * (du * decay * sigmoid(ag))[:cu[-1]].sum(0) * sigmoid(ap)
    for k in ("dx", "dx_gate", "dz", "da_gate"):
        if k in out:
            out[k][cu[-1]:] = np.nan
    return out
