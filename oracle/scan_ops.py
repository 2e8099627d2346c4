"""fp64 oracle for the selective state space scan -- TEST INFRASTRUCTURE ONLY.

    d_t = softplus(dt + bias) (or dt + bias),  a_t = exp(d_t A),  A = -exp(A_log)
    h_t = a_t h_{t-1} + d_t x_t B_t,  y_t = (sum_s h_t C_t + D x_t) silu(z_t)

Plain numpy in float64, token by token.  `walk` and `walk_back` take the steps
and decays as arrays, so that a test can also run them on magnitudes (every
input's absolute value) for an error bound.
"""
import numpy as np

from .layer_ops import _f64, silu


def softplus(v):
    return np.logaddexp(0.0, v)


def sigmoid(v):
    return np.exp(-np.logaddexp(0.0, -v))


def spread(v, C):
    """[T, G, S] of the groups as [T, C, S] of their channels."""
    return np.repeat(v, C // v.shape[1], axis=1)


def walk(d, A, x, B, C, h0):
    """States h [L, C, S] of one sequence from d, x [L, C], A [C, S], B, C [L, C, S], h0 [C, S]."""
    h = np.zeros(B.shape)
    s = h0
    for t in range(len(d)):
        s = np.exp(d[t][:, None] * A) * s + (d[t] * x[t])[:, None] * B[t]
        h[t] = s
    return h


def walk_back(d, A, x, B, C, h0, h, e, gT, A_sum=None):
    """Gradients of sum <e, sum_s h C> + <gT, last h>: dict of dx, dd, dB, dC [L, C, S] (per
    channel), dA [C, S], dh0.  A_sum: the A in the products outside the decays."""
    A_sum = A if A_sum is None else A_sum
    g = gT
    out = dict(dx=np.zeros(d.shape), dd=np.zeros(d.shape), dB=np.zeros(B.shape), dC=np.zeros(B.shape), dA=np.zeros(A.shape))
    for t in range(len(d) - 1, -1, -1):
        old = h[t - 1] if t else h0
        a = np.exp(d[t][:, None] * A)
        g = g + e[t][:, None] * C[t]
        out["dC"][t] = e[t][:, None] * h[t]
        out["dB"][t] = g * (d[t] * x[t])[:, None]
        u = (g * B[t]).sum(-1)
        w = g * a * old
        out["dx"][t] = d[t] * u
        out["dd"][t] = x[t] * u + (w * A_sum).sum(-1)
        out["dA"] += w * d[t][:, None]
        g = a * g
    out["dh0"] = g
    return out


def _inputs(x, dt, A_log, B, C, D, z, dt_bias, dt_softplus):
    x, dt, A_log, B, C, D, z, dt_bias = map(_f64, (x, dt, A_log, B, C, D, z, dt_bias))
    ch = x.shape[1]
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    d = softplus(raw) if dt_softplus else raw
    return x, raw, d, -np.exp(A_log), spread(B, ch), spread(C, ch), np.zeros(ch) if D is None else D, z


def selective_scan(x, dt, A_log, B, C, cu, D=None, z=None, dt_bias=None, init_state=None, dt_softplus=True):
    """(y [T, channels], final states [N, channels, S]); rows of y that no sequence covers are NaN."""
    x, _, d, A, B, C, D, z = _inputs(x, dt, A_log, B, C, D, z, dt_bias, dt_softplus)
    N = len(cu) - 1
    y = np.full(x.shape, np.nan)
    fin = np.zeros((N,) + A.shape) if init_state is None else _f64(init_state).copy()
    for n in range(N):
        s = slice(int(cu[n]), int(cu[n + 1]))
        if s.stop == s.start:
            continue
        h = walk(d[s], A, x[s], B[s], C[s], fin[n])
        y[s] = (h * C[s]).sum(-1) + D * x[s]
        fin[n] = h[-1]
    return (y if z is None else y * silu(z)), fin


def selective_scan_bwd(x, dt, A_log, B, C, cu, d_out, D=None, z=None, dt_bias=None, init_state=None, d_final_state=None,
                       dt_softplus=True, magnitude=False):
    """Gradients as gdn_selective_scan_bwd returns them; magnitude: every product with its
    absolute value, an upper bound of the sums' terms."""
    G = B.shape[1]
    x, raw, d, A, B, C, D, z = _inputs(x, dt, A_log, B, C, D, z, dt_bias, dt_softplus)
    dy = _f64(d_out)
    N, S = len(cu) - 1, A.shape[1]
    h0 = np.zeros((N,) + A.shape) if init_state is None else _f64(init_state)
    gT = np.zeros((N,) + A.shape) if d_final_state is None else _f64(d_final_state)
    p = None if z is None else sigmoid(z)
    e = dy if z is None else dy * z * p
    A_sum = A
    if magnitude:
        x, B, C, D, dy, e, h0, gT, A_sum = map(np.abs, (x, B, C, D, dy, e, h0, gT, A))
    T, ch = x.shape
    out = {k: np.full((T, ch), np.nan) for k in ("dx", "ddt", "dz")}
    out.update({k: np.full((T, G, S), np.nan) for k in ("dB", "dC")})
    out.update(dA_log=np.zeros(A.shape), dD=np.zeros(ch), ddt_bias=np.zeros(ch), d_init_state=np.zeros(h0.shape))
    for n in range(N):
        s = slice(int(cu[n]), int(cu[n + 1]))
        out["d_init_state"][n] = gT[n]
        if s.stop == s.start:
            continue
        h = walk(d[s], A, x[s], B[s], C[s], h0[n])
        r = walk_back(d[s], A, x[s], B[s], C[s], h0[n], h, e[s], gT[n], A_sum)
        out["dx"][s] = r["dx"] + D * e[s]
        ddt = r["dd"] * (sigmoid(raw[s]) if dt_softplus else 1.0)
        out["ddt"][s] = ddt
        out["dB"][s] = r["dB"].reshape(-1, G, ch // G, S).sum(2)
        out["dC"][s] = r["dC"].reshape(-1, G, ch // G, S).sum(2)
        if z is not None:
            slope = p[s] * (1.0 + z[s] * (1.0 - p[s]))
            if magnitude:  # the slope is a sum of two terms that cancel near z = -1.28
                slope = p[s] * (1.0 + np.abs(z[s]))
            out["dz"][s] = dy[s] * ((h * C[s]).sum(-1) + D * x[s]) * slope
        out["dA_log"] += r["dA"] * A_sum
        out["dD"] += (e[s] * x[s]).sum(0)
        out["ddt_bias"] += ddt.sum(0)
        out["d_init_state"][n] = r["dh0"]
    return out
