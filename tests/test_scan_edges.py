"""GPU checks of the selective scan and the q/k norm where single values leave the usual range,
and of the gradient on batches of many short sequences, against the fp64 oracles.  Bounds as in
test_scan.py and test_conv_qk_bwd.py."""
import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from oracle import layer_ops
from oracle import scan_ops as ref
from helpers import to_np
from test_conv_qk_bwd import turned, within
from test_scan import DEV, Case, bits, check

pytestmark = pytest.mark.gpu
INF = float("inf")


def check_forward(c, **kw):
    pool = c.h0.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, **kw, **c.args())
    want, fin = ref.selective_scan(cu=c.cu_list, init_state=c.h0, **kw, **c.args())
    absargs = {k: None if v is None else v.abs() if k in ("x", "B", "C", "D") else v for k, v in c.args().items()}
    mag, fmag = ref.selective_scan(cu=c.cu_list, init_state=c.h0.abs(), **kw, **dict(absargs, z=None))
    extra = 0.0
    if c.z is not None:
        mag, extra = mag * np.abs(ref.silu(to_np(c.z))), 6 + 2.4 * np.abs(to_np(c.z)).max()
    check(y, want, mag, c.units, c.dtype, extra)
    check(pool, fin, fmag, c.units, torch.float32)
    return y


def check_backward(c, **kw):
    """Every gradient against the oracle's, under test_scan.py's bound."""
    st = dict(init_state=c.h0, d_final_state=c.gT)
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, **st, **kw, **c.args())
    want = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, **st, **kw, **c.args())
    mag = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, magnitude=True, **st, **kw, **c.args())
    units = 3 * c.units + c.C + sum(c.lens) + (0 if c.z is None else 3 * (6 + 2.4 * np.abs(to_np(c.z)).max()))
    for k in want:
        if g[k] is not None:
            check(g[k], want[k], mag[k], units, torch.float32 if g[k].dtype == torch.float32 else c.dtype)
    return g


# ---------------------------------------------------------------- steps and decays out of range

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_steps(dtype):
    """dt = +inf: softplus is +inf, the state is forgotten and takes +inf B; dt = -inf: the token changes nothing."""
    dt = torch.zeros(3, 8, device=DEV, dtype=dtype)
    dt[1], dt[2] = INF, -INF
    one, bc = torch.ones(3, 8, device=DEV, dtype=dtype), torch.ones(3, 1, 8, device=DEV, dtype=dtype)
    s0 = torch.rand(3, 8, 8, device=DEV) + 1
    A = torch.zeros(8, 8, device=DEV)
    for call in ("update", "prompt"):
        st = s0.clone()
        if call == "update":
            y = gdn.gdn_selective_scan_update(one, dt, A, bc, bc, st)
        else:
            y = gdn.gdn_selective_scan_fwd(one, dt, A, bc, bc, torch.arange(4, dtype=torch.int32, device=DEV), state=st)
        assert torch.all(st[1] == INF) and torch.all(y[1] == INF), call
        assert torch.equal(st[2], s0[2]) and torch.isfinite(y[[0, 2]]).all() and torch.isfinite(st[0]).all(), call


@pytest.mark.parametrize("dtype,S,C", [(torch.float32, 16, 40), (torch.bfloat16, 32, 24), (torch.float32, 8, 72)])
def test_tokens_masked_by_their_step(dtype, S, C):
    """dt = -inf masks a token: d and its slope are 0, as in the formula."""
    c = Case([33, 5, 0, 18], C, 1, S, dtype, 31)
    c.units = c.error_units()
    c.dt[::3] = -INF
    check_forward(c)
    g = check_backward(c)
    assert torch.all(g["ddt"][:56:3] == 0)


@pytest.mark.parametrize("dtype,S,G,C", [(torch.float32, 16, 1, 40), (torch.bfloat16, 16, 2, 144), (torch.float32, 8, 1, 24), (torch.float32, 32, 1, 40), (torch.bfloat16, 64, 1, 24)])
def test_decays_beyond_fp32(dtype, S, G, C):
    """exp(A_log) past the largest fp32 value: such a state forgets at once; its gradients are 0 where the formula's
    are, also where sequences end inside a tile and where a step is 0."""
    c = Case([33, 0, 1, 70, 6], C, G, S, dtype, 32)
    c.units = c.error_units()
    c.A_log[::3, 1::4] = 88.6  # times log2(e) past it
    c.A_log[1::3, ::4] = 100.0
    c.A_log[2::3, 3::4] = 700.0
    check_forward(c)
    check_backward(c)
    c.dt[::4] = -INF
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype,S,G,CG", [(torch.float32, 16, 2, 24), (torch.bfloat16, 8, 2, 40), (torch.float32, 32, 3, 8), (torch.bfloat16, 64, 2, 16)])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_a_channels_parameters_stay_in_its_group(dtype, S, G, CG, bad):
    """A_log of channel 0 not a number: other channels' outputs and other groups' dB and dC have the bits they have without."""
    c = Case([21, 8, 3], G * CG, G, S, dtype, 33)
    st = dict(init_state=c.h0, d_final_state=c.gT)
    good = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, **st, **c.args())
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, **c.args())
    c.A_log[0] = bad
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, **st, **c.args())
    assert torch.equal(bits(gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, **c.args())[:, 1:]), bits(y[:, 1:]))
    for k in ("dx", "ddt", "dz", "dB", "dC", "d_init_state"):
        assert torch.equal(bits(g[k][:, 1:]), bits(good[k][:, 1:])), k
    for k in ("dA_log", "dD", "ddt_bias"):
        assert torch.equal(bits(g[k][1:]), bits(good[k][1:])), k


# ---------------------------------------------------------------- steps without softplus

@pytest.mark.parametrize("dtype,S,G,C,gate,bias", [(torch.float32, 16, 1, 72, True, True), (torch.bfloat16, 16, 2, 48, False, False),
                                                  (torch.bfloat16, 8, 1, 24, True, False), (torch.float32, 32, 1, 40, False, True),
                                                  (torch.float32, 64, 2, 32, True, False)])
def test_steps_without_softplus(dtype, S, G, C, gate, bias):
    """dt (+ dt_bias) taken as it is, prompts, single tokens and the gradient.  Here d is dt, exact, or one rounded sum:
    error_units counts more for it."""
    c = Case([33, 0, 1, 70, 16, 2], C, G, S, dtype, 34, gate=gate, bias=bias)
    c.dt = torch.rand(c.dt.shape, generator=torch.Generator().manual_seed(35)).to(dtype).to(DEV)
    if bias:
        c.bias = torch.rand(C, generator=torch.Generator().manual_seed(36)).to(DEV)
    d, A = to_np(c.dt) + (0 if not bias else to_np(c.bias)), np.exp(to_np(c.A_log))
    s = max((d[a:b].sum(0)[:, None] * A).max() for a, b in zip(c.cu_list, c.cu_list[1:]))
    c.units = 64 + 6 * max(c.lens) + 52 * min(40.0, s) + S / 4
    check_forward(c, dt_softplus=False)
    check_backward(c, dt_softplus=False)
    one = Case([1] * 9, C, G, S, dtype, 37, gate=gate, bias=bias)
    one.dt = c.dt[:9]
    a, b = one.h0.clone(), one.h0.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=one.cu, state=a, dt_softplus=False, **one.args())
    z = gdn.gdn_selective_scan_update(state=b, dt_softplus=False, **one.args())
    assert torch.equal(bits(y), bits(z)) and torch.equal(bits(a), bits(b))


# ---------------------------------------------------------------- many short sequences

@pytest.mark.parametrize("dtype,S,G,lens", [
    (torch.float32, 8, 2, [(0, 1, 7, 8, 9, 16, 17, 3)[i % 8] for i in range(300)]),
    (torch.bfloat16, 16, 1, [(13, 0, 24, 1, 40)[i % 5] for i in range(200)]),
    (torch.float32, 8, 365, [130, 1, 0, 250, 8, 7, 128, 129, 16, 611]),    # 16 tiles a segment
    (torch.bfloat16, 16, 183, [130, 1, 0, 250, 8, 7, 128, 129, 16, 611]),
    (torch.bfloat16, 16, 40, [130, 1, 0, 250, 8, 7, 128, 129, 16, 611]),   # 8
    (torch.float32, 32, 12, [130, 1, 0, 250, 8, 7, 128, 129, 16, 611]),    # 4
    (torch.bfloat16, 64, 2, [130, 1, 0, 250, 8, 7, 128, 129, 16, 611])])   # 2
def test_backward_of_sequences_of_every_length(dtype, S, G, lens):
    """Every sequence's states in a place of their own: the workspace filled with NaN changes nothing."""
    c = Case(lens, 8 * G, G, S, dtype, 38, slow=True)
    c.units = c.error_units()
    g = check_backward(c)
    shape = gdn.ScanShape(len(lens), sum(lens), 8 * G, G, S, int(dtype == torch.bfloat16), 1, 8 * G, 8 * G, 8 * G, G * S, G * S)
    ws = torch.full((gdn.lib().gdn_selective_scan_bwd_workspace_size(shape),), 255, dtype=torch.uint8, device=DEV)
    again = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, workspace=ws, **c.args())
    for k in g:
        assert torch.equal(bits(g[k]), bits(again[k])), k


# ---------------------------------------------------------------- q/k norm

@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("scale", [1.0, 1e-13, 1e-16, 1e-18])
def test_qk_gradient_of_small_rows_without_eps(norm, scale):
    """eps = 0 takes rows of any size: r^3 is past fp32 from rows of about 1e-13 down, the gradient is not."""
    gen = torch.Generator().manual_seed(41)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T, HQ, HK, d, rd = 7, 3, 2, 64, 32
    q, k, dq, dk = (rn(T, H, d).to(DEV) for H in (HQ, HK, HQ, HK))
    q, k = q * scale, k * scale
    w = (1 + 0.1 * rn(d)).to(DEV) if norm == "rms" else None
    th = rn(T, rd // 2)
    cos, sin = th.cos().to(DEV), th.sin().to(DEV)
    kw = dict(norm=norm, eps=0.0)
    out = gdn.gdn_qk_norm_rope(q, k, cos, sin, q_weight=w, k_weight=w, **kw)
    g = gdn.gdn_qk_norm_rope_bwd(q, k, cos, sin, dq, dk, q_weight=w, k_weight=w, **kw)
    aw, share = (1.0 if w is None else np.abs(to_np(w))), (1.0 / d if norm == "rms" else 1.0)
    for x, y, do, dx, dw in ((q, out[0], dq, g["dq"], g["dq_weight"]), (k, out[1], dk, g["dk"], g["dk_weight"])):
        r, ax = layer_ops._scale(to_np(x), norm, 0.0), np.abs(to_np(x))
        within(y, layer_ops.norm_rope(x, w, cos, sin, **kw), turned(ax * r * aw, cos, sin, False), d + 16, torch.float32)
        want, want_w = layer_ops.norm_rope_bwd(x, w, cos, sin, do, **kw)
        back = turned(np.abs(to_np(do)), cos, sin, False)
        ag = back * aw
        within(dx, want, r * ag + ax * r ** 3 * share * (ag * ax).sum(-1, keepdims=True), 3 * d + 32, torch.float32)
        if w is not None:
            within(dw, want_w, (back * ax * r).sum((0, 1)), 3 * d + 32 + T * x.shape[1], torch.float32)
