"""fp64 oracle for the ops around the Gated DeltaNet recurrence -- TEST INFRASTRUCTURE ONLY.

Only tests/, __graft_entry__.smoke() and bench.py's CPU baseline may use this
module; the library never does.

These are the next steps either side of the recurrent kernel in a GDN layer:
the gate activations that produce (g, beta) from the layer's projections,
the short causal depthwise conv (with its per-sequence conv state cache)
applied to the q/k/v projections before the recurrence, and the gated
RMSNorm applied to the recurrence's output.  The pages name them as part of
what the unified model carries over (A_log kept in fp32 through the trainer's
bf16 wrapping; the serving engine's conv state and SSM state caches reused
unchanged: "Defending Against the Training-Inference Numeric Mismatch in RL
(Especially Linear Attention)", sections 3.1 and 3.2); their formulas are
the standard Gated DeltaNet layer's:

    g    = -exp(A_log[h]) * softplus(a + dt_bias[h])         beta = sigmoid(b)
    conv: y[t, c] = silu( sum_i w[c, i] * xw[t + i, c] + bias[c] ),  i = 0..W-1,
          xw = (conv state: the W-1 input rows before the sequence) ++ (the sequence's rows)
    norm: y = o / sqrt(mean(o^2) + eps) * weight * silu(z)     (per token and head, over dv)

Plain numpy in float64; library primitives only (exp, logaddexp, sqrt).
"""
import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        import torch
        x = x.detach().to("cpu").to(torch.float64).numpy()
    return np.asarray(x, dtype=np.float64)


def gates(a, b, A_log, dt_bias):
    """(g, beta) from the raw projections a, b [T, HV] and per-head A_log, dt_bias [HV]."""
    a, b, A_log, dt_bias = map(_f64, (a, b, A_log, dt_bias))
    g = -np.exp(A_log)[None, :] * np.logaddexp(0.0, a + dt_bias[None, :])
    beta = 1.0 / (1.0 + np.exp(-b))
    return g, beta


def silu(x):
    return x / (1.0 + np.exp(-x))


def gated_rmsnorm(o, z, weight, eps=1e-6):
    """y[t, h, :] = o / sqrt(mean(o^2) + eps) * weight * silu(z) over the last axis."""
    o, z, weight = map(_f64, (o, z, weight))
    r = np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps)
    return o / r * weight * silu(z)


def causal_conv1d(x, w, cu_seqlens, bias=None, conv_state=None, activation=True):
    """Depthwise causal conv over packed varlen x [T, C] with taps w [C, W].

    conv_state [N, W-1, C] holds, per sequence, the W-1 input rows before it
    (zeros when None).  Returns (y [T, C], final conv state [N, W-1, C]): the
    last W-1 rows of (conv state ++ the sequence's inputs).
    """
    x, w, bias, conv_state = map(_f64, (x, w, bias, conv_state))
    cu = [int(c) for c in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    T, C = x.shape
    W = w.shape[1]
    N = len(cu) - 1
    y = np.zeros((T, C))
    final = np.zeros((N, W - 1, C))
    for n in range(N):
        a, e = cu[n], cu[n + 1]
        past = np.zeros((W - 1, C)) if conv_state is None else conv_state[n]
        xw = np.concatenate([past, x[a:e]], axis=0)  # [W-1 + L, C]
        for t in range(e - a):
            acc = np.zeros(C)
            for i in range(W):
                acc = acc + w[:, i] * xw[t + i]
            if bias is not None:
                acc = acc + bias
            y[a + t] = silu(acc) if activation else acc
        final[n] = xw[len(xw) - (W - 1):]
    return y, final


def causal_conv1d_update(x, w, conv_state, state_indices=None, bias=None, activation=True):
    """One decode token per sequence: x [B, C]; conv_state [slots, W-1, C] updated
    (returned as a copy); a negative slot skips the sequence (its y row stays 0)."""
    x, w, bias, conv_state = map(_f64, (x, w, bias, conv_state))
    B, C = x.shape
    W = w.shape[1]
    st = conv_state.copy()
    idx = list(range(B)) if state_indices is None else [int(i) for i in state_indices]
    y = np.zeros((B, C))
    for b in range(B):
        s = idx[b]
        if s < 0:
            continue
        xw = np.concatenate([st[s], x[b:b + 1]], axis=0)  # [W, C]
        acc = np.zeros(C)
        for i in range(W):
            acc = acc + w[:, i] * xw[i]
        if bias is not None:
            acc = acc + bias
        y[b] = silu(acc) if activation else acc
        st[s] = xw[1:]
    return y, st


def causal_conv1d_bwd(x, w, cu_seqlens, d_y, bias=None, init_state=None, d_final_state=None, activation=True):
    """Gradients of causal_conv1d for sum <d_y, y> + <d_final_state, final state>: dict dx
    [T, C] (NaN where no sequence is), dweight [C, W], dbias [C], d_init_state [N, W-1, C]."""
    x, w, bias, d_y, h0, dhT = map(_f64, (x, w, bias, d_y, init_state, d_final_state))
    cu = [int(c) for c in cu_seqlens]
    (T, C), W, N = x.shape, w.shape[1], len(cu) - 1
    out = dict(dx=np.full((T, C), np.nan), dweight=np.zeros((C, W)), dbias=np.zeros(C), d_init_state=np.zeros((N, W - 1, C)))
    for n in range(N):
        a, e = cu[n], cu[n + 1]
        rows = np.concatenate([np.zeros((W - 1, C)) if h0 is None else h0[n], x[a:e]])
        d_rows = np.zeros(rows.shape)
        if dhT is not None:
            d_rows[len(rows) - (W - 1):] += dhT[n]
        for t in range(e - a):
            pre = (w * rows[t:t + W].T).sum(1) + (0.0 if bias is None else bias)
            s = 1.0 / (1.0 + np.exp(-pre))
            p = d_y[a + t] * (s * (1.0 + pre * (1.0 - s)) if activation else 1.0)
            out["dbias"] += p
            out["dweight"] += p[:, None] * rows[t:t + W].T
            d_rows[t:t + W] += (p[:, None] * w).T
        out["d_init_state"][n] = d_rows[:W - 1]
        out["dx"][a:e] = d_rows[W - 1:]
    return out


def _turn(n, cos, sin, interleaved):
    """Rotation of n [T, H, d]'s first 2 * cos.shape[1] values by the tokens' angles [T, rd/2]."""
    half = cos.shape[1]
    out = n.copy()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = cos[:, None], sin[:, None]
    out[..., first] = n[..., first] * c - n[..., second] * s
    out[..., second] = n[..., second] * c + n[..., first] * s
    return out


def _scale(x, norm, eps):
    ss = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)


def norm_rope(x, weight, cos, sin, norm="rms", eps=1e-6, interleaved=False):
    """Normed and rotated heads of x [T, H, d]; cos, sin [T, rotary_dim / 2] of each token."""
    x, weight, cos, sin = map(_f64, (x, weight, cos, sin))
    return _turn(x * _scale(x, norm, eps) * (1.0 if weight is None else weight), cos, sin, interleaved)


def norm_rope_bwd(x, weight, cos, sin, d_out, norm="rms", eps=1e-6, interleaved=False):
    """(dx, dweight) of norm_rope for sum <d_out, out>."""
    x, weight, cos, sin, d_out = map(_f64, (x, weight, cos, sin, d_out))
    r = _scale(x, norm, eps)
    dn = _turn(d_out, cos, -sin, interleaved)
    g = dn * (1.0 if weight is None else weight)
    share = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    return r * g - x * r ** 3 * share * (g * x).sum(-1, keepdims=True), (dn * x * r).sum((0, 1))


def add_rmsnorm(s, weight, eps=1e-6):
    """The norm of s = x + residual (already rounded to its type) over the last axis, in float64."""
    s, weight = map(_f64, (s, weight))
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * weight


def group_scales(n, group):
    """max |n| / 448 of each `group` consecutive values of a row (0: the row), at least 2^-126."""
    d = n.shape[-1]
    per = group or d
    most = np.stack([np.abs(n[..., i:i + per]).max(-1) for i in range(0, d, per)], -1)
    return np.maximum(most / 448, 2.0 ** -126)


def add_rmsnorm_bwd(s, weight, d_out, d_residual_out=None, eps=1e-6, magnitude=False):
    """(dx, dweight); magnitude: sums over their terms' absolute values."""
    s, weight, dy = map(_f64, (s, weight, d_out))
    res = 0.0 if d_residual_out is None else _f64(d_residual_out)
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    if magnitude:
        s, weight, dy, res = np.abs(s), np.abs(weight), np.abs(dy), np.abs(res)
    g = dy * weight
    second = s * r ** 3 * (g * s).mean(-1, keepdims=True)
    dx = r * g + (second if magnitude else -second) + res
    return dx, (dy * s * r).reshape(-1, s.shape[-1]).sum(0)
