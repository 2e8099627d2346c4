"""GPU parity and gradients of the RMSNorm with the residual's addition against fp64
(oracle/layer_ops.py), and one layer around the gated linear recurrence end to end.

Tolerances, in units of u = 2^-24: the sum of d squares carries at most d roundings, its root half of
them, the hardware's reciprocal root and the products 10 more: (d / 2 + 10) u of a value.  A scale is one of
the values over 448, two roundings more.  In 8 bits a value is off by half a step of e4m3, 2^-4 of it, or
2^-10 of the scale among the smallest (steps of 2^-9), after its own (d / 2 + 16) u.  The gradient's
mean of g s carries 2 d roundings and r^3 three halves of d: (3 d + 32) u of its terms' magnitudes; dweight's
sum over T rows adds T.  A bf16 output adds its own rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from oracle import layer_ops
from oracle import linrec_ops
from helpers import BF16_ROUND, normwise, to_np
from test_linrec import BF, DEV, F32, U, bits

pytestmark = pytest.mark.gpu


def inputs(rows, d, dtype, seed, strided=False):
    gen = torch.Generator().manual_seed(seed)

    def wide(by=1.0):
        v = (torch.randn(rows, d + (24 if strided else 0), generator=gen) * by).to(dtype).to(DEV)
        return v[:, 8:-16] if strided else v

    return wide(), wide(2.0), (1 + 0.1 * torch.randn(d, generator=gen)).to(DEV), torch.randn(rows, d, generator=gen).to(dtype).to(DEV), \
        torch.randn(rows, d, generator=gen).to(dtype).to(DEV)


def within(got, want, mag, units, dtype):
    err = np.abs(to_np(got) - want)
    bound = units * U * mag + (BF16_ROUND if dtype == BF else U) * np.abs(want) + 1e-30
    assert np.all(err <= bound), (err / bound).max()


# widths: one lane, part of a warp, whole warps, several chunks a thread, several warps, the widest
SIZES = [(BF, 5, 8), (BF, 37, 72), (F32, 3, 4), (F32, 70, 200), (BF, 9, 1024), (BF, 33, 1032), (F32, 10, 1160), (BF, 4, 4096), (F32, 3, 4100), (BF, 7, 8192),
         (F32, 2, 8196), (BF, 3, 16384), (F32, 3, 16384), (BF, 1, 2056), (BF, 700, 264)]


@pytest.mark.parametrize("dtype,rows,d", SIZES)
@pytest.mark.parametrize("residual,strided", [(True, False), (True, True), (False, True)])
def test_forward_vs_oracle(dtype, rows, d, residual, strided):
    x, r, w, _, _ = inputs(rows, d, dtype, 3, strided)
    y, s = gdn.gdn_add_rmsnorm(x, w, residual=r if residual else None)
    if residual:
        assert torch.equal(bits(s), bits(x + r))
    else:
        assert s is None
    want = layer_ops.add_rmsnorm(s if residual else x, w)
    within(y, want, np.abs(want), d / 2 + 10, dtype)


@pytest.mark.parametrize("dtype,rows,d", SIZES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_fp8_vs_oracle(dtype, rows, d, group):
    x, r, w, _, _ = inputs(rows, d, dtype, 4)
    if rows > 2:
        x[1], r[1] = 0, 0  # a row of zeros
    q, scales, s = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=group)
    assert q.dtype == torch.float8_e4m3fn and torch.equal(bits(s), bits(x + r))
    n = layer_ops.add_rmsnorm(s, w)
    k = layer_ops.group_scales(n, group)
    assert scales.shape == k.shape
    within(scales, k, k, d / 2 + 12, F32)
    per = group or d
    each = np.repeat(to_np(scales), per, axis=1)[:, :d]
    err = np.abs(to_np(q.float()) * each - n)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * each) + (d / 2 + 16) * U * np.abs(n))
    # as the definition has it, from the same values in fp32: the kernel's norm in the type fp32 has those bits
    if dtype == F32:
        y, _ = gdn.gdn_add_rmsnorm(x, w, residual=r)
        wide = torch.from_numpy(each).float().to(DEV)
        step = (y / wide).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert (step.view(torch.uint8) != q.view(torch.uint8)).float().mean() < 1e-3  # a division and a product by the reciprocal differ next to a border


@pytest.mark.parametrize("dtype,rows,d", SIZES)
@pytest.mark.parametrize("residual,strided", [(True, False), (False, True)])
def test_backward_vs_oracle(dtype, rows, d, residual, strided):
    _, s, w, dy, dr = inputs(rows, d, dtype, 5, strided)
    g = gdn.gdn_add_rmsnorm_bwd(s, w, dy, d_residual_out=dr if residual else None)
    kw = dict(d_residual_out=dr if residual else None)
    dx, dw = layer_ops.add_rmsnorm_bwd(s, w, dy, **kw)
    mx, mw = layer_ops.add_rmsnorm_bwd(s, w, dy, magnitude=True, **kw)
    within(g["dx"], dx, mx, 3 * d + 32, dtype)
    within(g["dweight"], dw, mw, 3 * d + 32 + rows, F32)
    again = gdn.gdn_add_rmsnorm_bwd(s, w, dy, workspace=torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV), **kw)
    assert torch.equal(bits(again["dx"]), bits(g["dx"])) and torch.equal(bits(again["dweight"]), bits(g["dweight"]))


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 4096), (F32, 2060)])
def test_many_rows_have_the_bits_of_each_alone(dtype, d):
    rows = 3001
    x, r, w, dy, dr = inputs(rows, d, dtype, 6)
    y, s = gdn.gdn_add_rmsnorm(x, w, residual=r)
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=64)
    q0, k0, _ = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=0)
    g = gdn.gdn_add_rmsnorm_bwd(s, w, dy, d_residual_out=dr)
    for i in (0, 1, 7, 1500, 3000):
        t = slice(i, i + 1)
        y1, s1 = gdn.gdn_add_rmsnorm(x[t], w, residual=r[t])
        assert torch.equal(bits(y1), bits(y[t])) and torch.equal(bits(s1), bits(s[t]))
        q1, k1, _ = gdn.gdn_add_rmsnorm_fp8(x[t], w, residual=r[t], group=64)
        assert torch.equal(q1.view(torch.uint8), q[t].view(torch.uint8)) and torch.equal(k1, k[t])
        q1, k1, _ = gdn.gdn_add_rmsnorm_fp8(x[t], w, residual=r[t], group=0)
        assert torch.equal(q1.view(torch.uint8), q0[t].view(torch.uint8)) and torch.equal(k1, k0[t])
        assert torch.equal(bits(gdn.gdn_add_rmsnorm_bwd(s[t], w, dy[t], d_residual_out=dr[t])["dx"]), bits(g["dx"][t]))
    dx, dw = layer_ops.add_rmsnorm_bwd(s, w, dy, dr)
    _, mw = layer_ops.add_rmsnorm_bwd(s, w, dy, dr, magnitude=True)
    within(g["dweight"], dw, mw, 3 * d + 32 + rows, F32)


@pytest.mark.parametrize("dtype,d", [(BF, 2048), (F32, 520)])
def test_in_place(dtype, d):
    x, r, w, dy, dr = inputs(21, d, dtype, 7)
    y, s = gdn.gdn_add_rmsnorm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    gdn.gdn_add_rmsnorm(a, w, residual=b, out=a, residual_out=b)
    assert torch.equal(bits(a), bits(y)) and torch.equal(bits(b), bits(s))
    a, b = x.clone(), r.clone()
    gdn.gdn_add_rmsnorm(a, w, residual=b, out=b, residual_out=a)
    assert torch.equal(bits(b), bits(y)) and torch.equal(bits(a), bits(s))
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r)
    b = r.clone()
    q2, k2, s2 = gdn.gdn_add_rmsnorm_fp8(x, w, residual=b, residual_out=b)
    assert s2 is b and torch.equal(bits(b), bits(s)) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(k, k2)
    g = gdn.gdn_add_rmsnorm_bwd(s, w, dy, d_residual_out=dr)["dx"]
    for which in range(3):
        v = [s.clone(), dy.clone(), dr.clone()]
        got = gdn.gdn_add_rmsnorm_bwd(v[0], w, v[1], d_residual_out=v[2], dx=v[which])["dx"]
        assert got is v[which] and torch.equal(bits(got), bits(g))


@pytest.mark.parametrize("dtype,d,group", [(BF, 72, 32), (F32, 72, 0), (BF, 4096, 128), (F32, 1160, 64)])
def test_fp8_out_at_8_bytes(dtype, d, group):
    """y in 8 bits needs 8-byte alignment only."""
    x, r, w, _, _ = inputs(5, d, dtype, 17)
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=group)
    whole = torch.full((5 * d + 24,), 0x55, dtype=torch.uint8, device=DEV)
    out = whole[8:8 + 5 * d].view(torch.float8_e4m3fn).view(5, d)
    got, k2, _ = gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=group, out=out)
    assert got is out and out.data_ptr() % 16 == 8
    assert torch.equal(out.view(torch.uint8), q.view(torch.uint8)) and torch.equal(k, k2)
    assert torch.all(whole[:8] == 0x55) and torch.all(whole[8 + 5 * d:] == 0x55)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, group=group, out=whole[4:4 + 5 * d].view(torch.float8_e4m3fn).view(5, d))


def test_no_rows_and_leading_dimensions():
    w = torch.ones(64, device=DEV)
    for shape in ((0, 64), (2, 0, 64)):
        x = torch.empty(shape, device=DEV)
        y, s = gdn.gdn_add_rmsnorm(x, w, residual=x)
        assert y.shape == s.shape == x.shape
        q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w)
        assert q.shape == x.shape and k.shape == x.shape[:-1] + (1,)
        assert torch.all(gdn.gdn_add_rmsnorm_bwd(x, w, x)["dweight"] == 0)
    x, r, w, dy, _ = inputs(12, 200, BF, 8)
    y, s = gdn.gdn_add_rmsnorm(x, w, residual=r)
    y3, s3 = gdn.gdn_add_rmsnorm(x.view(3, 4, 200), w, residual=r.view(3, 4, 200))
    assert y3.shape == (3, 4, 200) and torch.equal(bits(y3.view(12, 200)), bits(y)) and torch.equal(bits(s3.view(12, 200)), bits(s))
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x.view(3, 4, 200), w, residual=r.view(3, 4, 200))
    assert q.shape == (3, 4, 200) and k.shape == (3, 4, 2)
    y1, _ = gdn.gdn_add_rmsnorm(x[0], w, residual=r[0])
    assert y1.shape == (200,) and torch.equal(bits(y1), bits(y[0]))


def test_values_far_out():
    """A row with a NaN or an infinity is lost, its neighbours are not; eps = 0 takes small rows; large rows stay finite."""
    x, _, w, dy, _ = inputs(6, 256, F32, 9)
    y0, _ = gdn.gdn_add_rmsnorm(x, w)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    y, _ = gdn.gdn_add_rmsnorm(x, w)
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w, group=128)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 200]) and torch.equal(bits(y[[0, 3, 4, 5]]), bits(y0[[0, 3, 4, 5]]))
    assert torch.isnan(q[1].float()).all() and torch.isnan(q[2].float()[200]) and torch.isfinite(q[[0, 3, 4, 5]].float()).all() and torch.isfinite(k).all()
    for by in (1e-16, 1e16):
        s = inputs(4, 256, F32, 10)[0] * by
        want = layer_ops.add_rmsnorm(s, w, 0.0)
        y, _ = gdn.gdn_add_rmsnorm(s, w, eps=0.0)
        within(y, want, np.abs(want), 138, F32)
        d4 = dy[:4].contiguous()
        dx, dw = layer_ops.add_rmsnorm_bwd(s, w, d4, eps=0.0)
        mx, mw = layer_ops.add_rmsnorm_bwd(s, w, d4, eps=0.0, magnitude=True)
        g = gdn.gdn_add_rmsnorm_bwd(s, w, d4, eps=0.0)
        within(g["dx"], dx, mx, 3 * 256 + 32, F32)
        within(g["dweight"], dw, mw, 3 * 256 + 36, F32)


@pytest.mark.parametrize("dtype,d", [(F32, 256), (BF, 512), (F32, 8196)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_fp8_values_go_by_the_stored_scale(dtype, d, group):
    """Groups whose scale is the smallest one, 2^-126: y is still value / scale.  Rows whose sum of squares is past fp32 have a norm of 0."""
    x = torch.randn(4, d, generator=torch.Generator().manual_seed(15))
    x[0, 3], x[1, 5], x[2], x[3] = float("inf"), 1e20, x[2] * 1e-20, x[3] * 1e-24
    x[2:, 0] = 1e17  # r: sqrt(d) 1e-17; values of 1e-35 to 1e-39 behind it
    x = x.to(dtype).to(DEV)
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(16))).to(DEV)
    q, k, _ = gdn.gdn_add_rmsnorm_fp8(x, w, eps=0.0, group=group)
    q, least = q.float(), 2.0 ** -126
    assert torch.isnan(q[0, 3]) and torch.all(q[0, 4:] == 0) and torch.all(q[0, :3] == 0) and torch.all(q[1] == 0) and torch.all(k[:2] == least)
    n = layer_ops.add_rmsnorm(x[2:], w, 0.0)
    want = layer_ops.group_scales(n, group)
    assert group == 0 or np.any(want == least)
    within(k[2:], want, want, d / 2 + 12, F32)
    each = np.repeat(want, group or d, axis=1)[:, :d]
    # half a step of e4m3, and the value's own error (module docstring); below 2^-126 the product s w r may lose half of 2^-149
    err = np.abs(to_np(q[2:]) * each - n)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * each) + (d + 28) * U * np.abs(n) + 2.0 ** -149)


def test_offsets_past_2_31():
    ld = 48 << 20
    wide = torch.zeros(50, ld, dtype=BF, device=DEV)
    x, r, w, dy, dr = inputs(50, 64, BF, 11)
    wide[:, :64], wide[:, 64:128] = x, r
    assert 49 * ld > 2 ** 31
    y, s = gdn.gdn_add_rmsnorm(x, w, residual=r)
    y2, s2 = gdn.gdn_add_rmsnorm(wide[:, :64], w, residual=wide[:, 64:128])
    assert torch.equal(bits(y), bits(y2)) and torch.equal(bits(s), bits(s2))
    a, b = (gdn.gdn_add_rmsnorm_bwd(v, w, dy, d_residual_out=dr) for v in (x, wide[:, :64]))
    assert torch.equal(bits(a["dx"]), bits(b["dx"])) and torch.equal(bits(a["dweight"]), bits(b["dweight"]))


def test_captured_calls_and_other_streams():
    x, r, w, dy, dr = inputs(40, 512, BF, 12)
    x2, r2, _, dy2, dr2 = inputs(40, 512, BF, 13)
    run = lambda: (*gdn.gdn_add_rmsnorm(x, w, residual=r), *gdn.gdn_add_rmsnorm_fp8(x, w, residual=r)[:2], *gdn.gdn_add_rmsnorm_bwd(x, w, dy, d_residual_out=dr).values())  # noqa: E731
    first = [t.clone() for t in run()]
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    kw = dict(stream=other)
    got = (*gdn.gdn_add_rmsnorm(x, w, residual=r, **kw), *gdn.gdn_add_rmsnorm_fp8(x, w, residual=r, **kw)[:2],
           *gdn.gdn_add_rmsnorm_bwd(x, w, dy, d_residual_out=dr, **kw).values())
    other.synchronize()
    same = lambda u, v: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(u, v))  # noqa: E731
    assert same(got, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for a, b in ((x, x2), (r, r2), (dy, dy2), (dr, dr2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in out]
    assert same(replayed, run()) and not same(replayed, first)


def test_refused_tensors():
    x, w = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV)
    wide = torch.zeros(4, 130, device=DEV)
    for error, call in (
            (ValueError, lambda: gdn.gdn_add_rmsnorm(x, w[:32])), (TypeError, lambda: gdn.gdn_add_rmsnorm(x, w.bfloat16())),
            (ValueError, lambda: gdn.gdn_add_rmsnorm(x, w, residual=x[:2])), (TypeError, lambda: gdn.gdn_add_rmsnorm(x, w, residual=x.bfloat16())),
            (ValueError, lambda: gdn.gdn_add_rmsnorm(x.t().contiguous().t(), w)), (ValueError, lambda: gdn.gdn_add_rmsnorm(x, w, residual_out=x)),
            (TypeError, lambda: gdn.gdn_add_rmsnorm(x.half(), w)), (gdn.GdnError, lambda: gdn.gdn_add_rmsnorm(wide[:, :64], w)),
            (ValueError, lambda: gdn.gdn_add_rmsnorm(x, w, out=wide[:, :64])), (gdn.GdnError, lambda: gdn.gdn_add_rmsnorm(x, w, eps=-1.0)),
            (gdn.GdnError, lambda: gdn.gdn_add_rmsnorm_fp8(x, w, group=16)), (TypeError, lambda: gdn.gdn_add_rmsnorm_fp8(x, w, out=x)),
            (ValueError, lambda: gdn.gdn_add_rmsnorm_fp8(x, w, scales=x)), (ValueError, lambda: gdn.gdn_add_rmsnorm_bwd(x, w, x[:2])),
            (gdn.GdnError, lambda: gdn.gdn_add_rmsnorm(torch.zeros(4, 62, device=DEV), w[:62]))):
        with pytest.raises(error):
            call()
    assert gdn.gdn_add_rmsnorm(x, w)[0].shape == (4, 64)


# ---------------------------------------------------------------- a layer

def test_a_layer_prompt_tokens_and_gradient():
    """norm with residual -> projections -> conv -> gated recurrence -> output projection, as a model runs it: one prompt has the bits of
    prompt and single tokens, and the gradient is the fp64 layer's."""
    gen = torch.Generator().manual_seed(14)
    rn = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    lens, d, C, W = [70, 0, 41], 64, 96, 4
    T, cu_list = sum(lens), [0, 70, 70, 111]
    cu = torch.tensor(cu_list, dtype=torch.int32, device=DEV)
    x, res, nw = rn(T, d), rn(T, d), 1 + 0.1 * rn(d)
    proj, wo, cw, cb = rn(d, 4 * C) / 8, rn(C, d) / 10, rn(C, W) / 2, 0.1 * rn(C)
    ap = torch.log(torch.expm1(-torch.log(0.9 + 0.09 * torch.rand(C, generator=gen)) / 8)).to(DEV)

    def product(v, m):  # row by row: torch's sum over a dimension depends on how many rows there are
        return torch.stack([(row[:, None] * m).sum(0) for row in v])

    def layer(x, res, cu, conv, state, idx):
        n, s = gdn.gdn_add_rmsnorm(x, nw, residual=res)
        p = product(n, proj)
        c = gdn.gdn_causal_conv1d_fwd(p[:, :C].contiguous(), cw, cu, bias=cb, conv_state=conv, state_indices=idx, activation=False)
        y = gdn.gdn_linear_recurrence_fwd(c, p[:, C:2 * C], cu, a_param=ap, x_gate=p[:, 2 * C:3 * C], z=p[:, 3 * C:], state=state, state_indices=idx, activation="gelu")
        return product(y, wo) + s, (n, s, p, c, y)

    conv, state = torch.zeros(3, W - 1, C, device=DEV), torch.zeros(3, C, device=DEV)
    out, (n, s, p, c, y) = layer(x, res, cu, conv, state, None)
    # the third sequence: 30 tokens as a prompt, then one by one
    cv, st, idx = torch.zeros(2, W - 1, C, device=DEV), torch.zeros(2, C, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV)
    parts = [layer(x[70:100], res[70:100], torch.tensor([0, 30], dtype=torch.int32, device=DEV), cv, st, idx)[0]]
    for t in range(100, 111):
        n1, s1 = gdn.gdn_add_rmsnorm(x[t:t + 1], nw, residual=res[t:t + 1])
        p1 = product(n1, proj)
        c1 = gdn.gdn_causal_conv1d_update(p1[:, :C].contiguous(), cw, cv, state_indices=idx, bias=cb, activation=False)
        y1 = gdn.gdn_linear_recurrence_update(c1, p1[:, C:2 * C], st, state_indices=idx, a_param=ap, x_gate=p1[:, 2 * C:3 * C], z=p1[:, 3 * C:], activation="gelu")
        parts.append(product(y1, wo) + s1)
    assert torch.equal(bits(torch.cat(parts)), bits(out[70:])) and torch.equal(bits(st[1]), bits(state[2])) and torch.equal(bits(cv[1]), bits(conv[2]))

    # gradient of <out, do>
    do = rn(T, d)
    g = gdn.gdn_linear_recurrence_bwd(c, p[:, C:2 * C], cu, product(do, wo.t().contiguous()), a_param=ap, x_gate=p[:, 2 * C:3 * C], z=p[:, 3 * C:], activation="gelu")
    gc = gdn.gdn_causal_conv1d_bwd(p[:, :C].contiguous(), cw, cu, g["dx"], bias=cb, activation=False)
    dp = torch.cat([gc["dx"], g["da_gate"], g["dx_gate"], g["dz"]], 1)
    gn = gdn.gdn_add_rmsnorm_bwd(s, nw, product(dp, proj.t().contiguous()), d_residual_out=do)
    leaf = {k: v.double().requires_grad_() for k, v in dict(x=x, res=res, nw=nw, proj=proj, cw=cw, cb=cb, ap=ap, wo=wo).items()}
    s6 = leaf["x"] + leaf["res"]
    p6 = s6 / torch.sqrt(s6.square().mean(-1, keepdim=True) + 1e-6) * leaf["nw"] @ leaf["proj"]
    loss = (s6 * do.double()).sum()
    for lo, hi in zip(cu_list, cu_list[1:]):
        rows = torch.cat([p6.new_zeros(W - 1, C), p6[lo:hi, :C]])
        u = -8 * torch.nn.functional.softplus(leaf["ap"]) * torch.sigmoid(p6[lo:hi, C:2 * C])
        h = p6.new_zeros(C)
        for t in range(hi - lo):
            v = (rows[t:t + W] * leaf["cw"].t()).sum(0) + leaf["cb"]
            h = torch.exp(u[t]) * h + torch.sqrt(-torch.expm1(2 * u[t])) * v * torch.sigmoid(p6[lo + t, 2 * C:3 * C])
            loss = loss + (h * torch.nn.functional.gelu(p6[lo + t, 3 * C:], approximate="tanh") @ leaf["wo"] * do[lo + t].double()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    # each stage's bound is a few thousand u of its terms' magnitudes; five stages of sums of up to 100 mixed signs: 1e-4 of the largest value
    for got, k in ((gn["dx"], "x"), (gn["dx"], "res"), (gn["dweight"], "nw"), (gc["dweight"], "cw"), (gc["dbias"], "cb"), (g["da_param"], "ap")):
        assert normwise(to_np(got), to_np(want[k])) < 1e-4, k
    # and the recurrence itself against its oracle, on what the layer gave it
    ref, _ = linrec_ops.linear_recurrence(c, p[:, C:2 * C], cu_list, a_param=ap, x_gate=p[:, 2 * C:3 * C], z=p[:, 3 * C:], activation="gelu")
    assert normwise(to_np(y), ref) < 1e-5
