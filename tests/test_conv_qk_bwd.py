"""GPU parity of the conv's gradient and of the q/k norm with rotation and its gradient
against the fp64 oracle (oracle/layer_ops.py), and a run of the operators together.

Tolerances, u = 2^-24, in units of the sum of the terms' magnitudes M:
  * conv: pre is W + 1 fused multiply-adds; p = d_y act'(pre) adds at most 24 u (sigmoid through
    the hardware exponential and reciprocal, its slope a sum of two terms of one size) plus
    1.3 (W + 1) u M_pre of pre's own error; then W more products: dx within
    (2 W + 32 + 1.3 (W + 1) M_pre) u M; the sums over T tokens add T u.
  * q/k: the sum of d squares (d u), the root and four products (relative, 8 u), the rotation
    (two products and a sum, 3 u of |u cos| + |v sin|): (d + 16) u M; the gradient's
    dot product adds d u: (3 d + 32) u M; dweight adds one rounding per row.
A bf16 output adds 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from oracle import layer_ops as ref
from helpers import BF16_ROUND, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def rounding(dtype):
    return BF16_ROUND if dtype == torch.bfloat16 else U


def within(got, want, mag, units, dtype):
    got = to_np(got)
    ok = ~np.isnan(want)
    bound = units * U * mag[ok] + rounding(dtype) * np.abs(want[ok]) + 1e-30
    err = np.abs(got[ok] - want[ok])
    assert np.all(err <= bound), (err / bound).max()


# ---------------------------------------------------------------- conv gradient

CONV_LENS = [5, 0, 1, 2, 130, 3, 64, 0, 17]


@pytest.mark.parametrize("dtype,W,C", [(torch.bfloat16, 4, 520), (torch.float32, 4, 36), (torch.bfloat16, 2, 8), (torch.float32, 8, 1028),
                                       (torch.bfloat16, 3, 64), (torch.float32, 5, 12), (torch.bfloat16, 6, 16), (torch.float32, 7, 8),
                                       (torch.bfloat16, 8, 32)])
@pytest.mark.parametrize("full", [True, False])
def test_conv_backward_vs_oracle(dtype, W, C, full):
    gen = torch.Generator().manual_seed(W)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N, T = len(CONV_LENS), sum(CONV_LENS) + 2
    cu = np.concatenate([[0], np.cumsum(CONV_LENS)]).tolist()
    x, dy = rn(T, C).to(dtype).to(DEV), rn(T, C).to(dtype).to(DEV)
    x[T - 2:] = float("nan")
    w = (rn(C, W) / W ** 0.5).to(DEV)
    kw = {}
    if full:
        kw = dict(bias=(0.1 * rn(C)).to(DEV), init_state=rn(N, W - 1, C).to(dtype).to(DEV), d_final_state=rn(N, W - 1, C).to(dtype).to(DEV))
    g = gdn.gdn_causal_conv1d_bwd(x, w, torch.tensor(cu, dtype=torch.int32, device=DEV), dy, activation=full, **kw)
    want = ref.causal_conv1d_bwd(x, w, cu, dy, activation=full, **kw)
    absk = {k: v.abs() for k, v in kw.items()}
    mag = ref.causal_conv1d_bwd(x.abs(), w.abs(), cu, dy.abs() * 1.1, activation=False, **absk)
    pre, _ = ref.causal_conv1d(x.abs()[:T - 2], w.abs(), cu, bias=absk.get("bias"), conv_state=absk.get("init_state"), activation=False)
    units = 2 * W + 32 + 1.3 * (W + 1) * (pre.max() if full else 0)
    within(g["dx"], want["dx"], mag["dx"], units, dtype)
    within(g["d_init_state"], want["d_init_state"], mag["d_init_state"], units, dtype)
    within(g["dweight"], want["dweight"], mag["dweight"], units + T, torch.float32)
    if full:
        within(g["dbias"], want["dbias"], mag["dbias"], units + T, torch.float32)
    else:
        assert g["dbias"] is None


def test_conv_backward_long_batches_sampled_and_repeated():
    """More tokens than ranges: every range border against the sums of a two-piece split."""
    T, C, W = 5000, 1024, 4
    gen = torch.Generator().manual_seed(9)
    x, dy = (torch.randn(T, C, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    w, b = torch.randn(C, W, generator=gen).to(DEV) / 2, torch.randn(C, generator=gen).to(DEV)
    cu = torch.tensor([0, 1700, 1701, 5000], dtype=torch.int32, device=DEV)
    g = gdn.gdn_causal_conv1d_bwd(x, w, cu, dy, bias=b)
    again = gdn.gdn_causal_conv1d_bwd(x, w, cu, dy, bias=b)
    for k in g:
        assert torch.equal(bits(g[k]), bits(again[k])), k
    cols = slice(500, 508)
    want = ref.causal_conv1d_bwd(x[:, cols], w[cols], cu.tolist(), dy[:, cols], bias=b[cols])
    mag = ref.causal_conv1d_bwd(x[:, cols].abs(), w[cols].abs(), cu.tolist(), dy[:, cols].abs() * 1.1, bias=b[cols].abs(), activation=False)
    pre, _ = ref.causal_conv1d(x[:, cols].abs(), w[cols].abs(), cu.tolist(), bias=b[cols].abs(), activation=False)
    units = 2 * W + 32 + 1.3 * (W + 1) * pre.max()
    within(g["dx"][:, cols], want["dx"], mag["dx"], units, torch.bfloat16)
    within(g["dweight"][cols], want["dweight"], mag["dweight"], units + T, torch.float32)
    within(g["dbias"][cols], want["dbias"], mag["dbias"], units + T, torch.float32)
    # a sequence's rows of dx do not depend on the batch
    alone = gdn.gdn_causal_conv1d_bwd(x[1701:], w, torch.tensor([0, 3299], dtype=torch.int32, device=DEV), dy[1701:], bias=b)
    assert torch.equal(bits(alone["dx"]), bits(g["dx"][1701:]))


def test_conv_backward_without_tokens():
    x = torch.empty(0, 16, device=DEV)
    w = torch.randn(16, 4, device=DEV)
    dT = torch.randn(3, 3, 16, device=DEV)
    g = gdn.gdn_causal_conv1d_bwd(x, w, torch.zeros(4, dtype=torch.int32, device=DEV), x, bias=w[:, 0].contiguous(), d_final_state=dT)
    assert torch.equal(g["d_init_state"], dT) and torch.all(g["dweight"] == 0) and torch.all(g["dbias"] == 0)
    x = torch.full((7, 16), float("nan"), device=DEV)  # padding only
    g = gdn.gdn_causal_conv1d_bwd(x, w, torch.zeros(4, dtype=torch.int32, device=DEV), x, bias=w[:, 0].contiguous(), d_final_state=dT)
    assert torch.equal(g["d_init_state"], dT) and torch.all(g["dweight"] == 0) and torch.all(g["dbias"] == 0)


# ---------------------------------------------------------------- q/k norm with rotation

QK = [(torch.bfloat16, 5, 4, 2, 128, 128, "l2", False), (torch.bfloat16, 37, 3, 1, 256, 64, "rms", False),
      (torch.float32, 9, 6, 3, 80, 80, "rms", True), (torch.float32, 1, 1, 1, 256, 256, "l2", True),
      (torch.bfloat16, 300, 1, 5, 8, 0, "rms", False), (torch.bfloat16, 64, 16, 0, 96, 32, "rms", True),
      (torch.float32, 33, 2, 7, 4, 0, "l2", False), (torch.bfloat16, 3000, 5, 3, 72, 64, "rms", False),
      (torch.bfloat16, 11, 8, 8, 192, 192, "rms", True), (torch.float32, 2600, 2, 2, 20, 16, "rms", False)]


class QkCase:
    def __init__(self, dtype, T, HQ, HK, d, rd, norm, seed=3):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        wide = rn(T, (HQ + 2 * HK) * d + 16).to(dtype).to(DEV)
        self.q = wide[:, 8:8 + HQ * d].unflatten(1, (HQ, d)) if dtype == torch.bfloat16 else wide[:, 4:4 + HQ * d].unflatten(1, (HQ, d))
        self.k = wide[:, 8 + HQ * d:8 + (HQ + HK) * d].reshape(T, HK, d)
        P = 97
        th = rn(P, rd // 2) * 3
        self.cos, self.sin = th.cos().to(DEV), th.sin().to(DEV)
        self.pos = torch.randint(0, P, (T,), generator=gen, dtype=torch.int32).to(DEV)
        self.qw = (1 + 0.2 * rn(d)).to(DEV) if norm == "rms" else None
        self.kw = (1 + 0.2 * rn(d)).to(DEV) if norm == "rms" and HK else None
        self.dq, self.dk = rn(T, HQ, d).to(dtype).to(DEV), rn(T, HK, d).to(dtype).to(DEV)


def turned(n, cs, sn, inter):
    """|u cos| + |v sin| and |v cos| + |u sin| of magnitudes n."""
    c, s = np.abs(to_np(cs)), np.abs(to_np(sn))
    return np.maximum(ref._turn(n, c, s, inter), ref._turn(n, c, -s, inter))


@pytest.mark.parametrize("dtype,T,HQ,HK,d,rd,norm,inter", QK)
def test_qk_norm_rope_vs_oracle(dtype, T, HQ, HK, d, rd, norm, inter):
    c = QkCase(dtype, T, HQ, HK, d, rd, norm)
    kw = dict(norm=norm, eps=1e-5, interleaved=inter)
    qo, ko = gdn.gdn_qk_norm_rope(c.q, c.k, c.cos, c.sin, positions=c.pos, q_weight=c.qw, k_weight=c.kw, **kw)
    g = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, positions=c.pos, q_weight=c.qw, k_weight=c.kw, **kw)
    cs, sn = c.cos[c.pos.long()], c.sin[c.pos.long()]
    for x, w, out, do, dx, dw in ((c.q, c.qw, qo, c.dq, g["dq"], g["dq_weight"]), (c.k, c.kw, ko, c.dk, g["dk"], g["dk_weight"])):
        if x.shape[1] == 0:
            assert out.shape == x.shape and dw is None
            continue
        r = ref._scale(to_np(x), norm, 1e-5)
        aw = 1.0 if w is None else np.abs(to_np(w))
        n = np.abs(to_np(x)) * r * aw
        within(out, ref.norm_rope(x, w, cs, sn, **kw), turned(n, cs, sn, inter), d + 16, dtype)
        want, want_w = ref.norm_rope_bwd(x, w, cs, sn, do, **kw)
        back = turned(np.abs(to_np(do)), cs, sn, inter)
        ag, ax = back * aw, np.abs(to_np(x))
        share = 1.0 / d if norm == "rms" else 1.0
        within(dx, want, r * ag + ax * r ** 3 * share * (ag * ax).sum(-1, keepdims=True), 3 * d + 32, dtype)
        if w is not None:
            within(dw, want_w, (back * ax * r).sum((0, 1)), 3 * d + 32 + T * x.shape[1], torch.float32)


def test_qk_rows_do_not_depend_on_the_batch_and_skipped_tokens_stay():
    c = QkCase(torch.bfloat16, 4000, 3, 2, 64, 32, "rms")
    args = dict(q_weight=c.qw, k_weight=c.kw)
    qo, ko = gdn.gdn_qk_norm_rope(c.q, c.k, c.cos, c.sin, positions=c.pos, **args)
    q1, k1 = gdn.gdn_qk_norm_rope(c.q[7:8], c.k[7:8], c.cos, c.sin, positions=c.pos[7:8], **args)
    assert torch.equal(bits(q1), bits(qo[7:8])) and torch.equal(bits(k1), bits(ko[7:8]))
    again = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, positions=c.pos, **args)
    once = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, positions=c.pos, **args)
    for k in again:
        assert torch.equal(bits(again[k]), bits(once[k])), k
    pos = c.pos.clone()
    pos[5], pos[3999] = -1, 97  # outside the tables
    out = [torch.full(t.shape, 9.0, dtype=torch.bfloat16, device=DEV) for t in (c.q, c.k, c.q, c.k)]
    gdn.gdn_qk_norm_rope(c.q, c.k, c.cos, c.sin, positions=pos, q_out=out[0], k_out=out[1], **args)
    g = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, positions=pos, dq=out[2], dk=out[3], **args)
    for t in out:
        assert torch.all(t[[5, 3999]] == 9) and not torch.any(torch.all(t[6:3999].flatten(1) == 9, 1))
    keep = torch.tensor([i for i in range(4000) if i not in (5, 3999)], device=DEV)
    want = ref.norm_rope_bwd(c.q[keep], c.qw, c.cos[c.pos[keep].long()], c.sin[c.pos[keep].long()], c.dq[keep])[1]
    assert np.abs(to_np(g["dq_weight"]) - want).max() <= 1e-4 * np.abs(want).max()


def test_qk_with_one_weight():
    c = QkCase(torch.bfloat16, 40, 3, 2, 64, 32, "rms")
    cs, sn = c.cos[c.pos.long()], c.sin[c.pos.long()]
    for kw in (dict(q_weight=c.qw), dict(k_weight=c.kw)):
        qo, ko = gdn.gdn_qk_norm_rope(c.q, c.k, c.cos, c.sin, positions=c.pos, **kw)
        g = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, positions=c.pos, **kw)
        for x, w, out, do, dx, dw in ((c.q, kw.get("q_weight"), qo, c.dq, g["dq"], g["dq_weight"]),
                                      (c.k, kw.get("k_weight"), ko, c.dk, g["dk"], g["dk_weight"])):
            want, want_w = ref.norm_rope_bwd(x, w, cs, sn, do)
            assert np.abs(to_np(out) - ref.norm_rope(x, w, cs, sn)).max() <= 2 * BF16_ROUND * np.abs(to_np(out)).max()
            assert np.abs(to_np(dx) - want).max() <= 2 * BF16_ROUND * np.abs(want).max()
            assert (dw is None) == (w is None)
            if w is not None:
                assert np.abs(to_np(dw) - want_w).max() <= 1e-4 * np.abs(want_w).max()


@pytest.mark.parametrize("inter", [False, True])
def test_qk_infinity_stays_in_its_pair(inter):
    # r = 0 in a row with an infinity: its finite values become 0, the infinity (and, rotated, its pair) NaN
    x = torch.randn(2, 1, 32, generator=torch.Generator().manual_seed(1)).to(DEV)
    x[0, 0, 20] = float("inf")  # not rotated
    x[1, 0, 3] = float("inf")   # rotated: pairs (3, 11) or (2, 3)
    th = torch.randn(2, 8, generator=torch.Generator().manual_seed(2)).to(DEV)
    out, _ = gdn.gdn_qk_norm_rope(x, x, th.cos(), th.sin(), interleaved=inter)
    assert torch.isnan(out[0, 0]).nonzero().flatten().tolist() == [20]
    assert torch.isnan(out[1, 0]).nonzero().flatten().tolist() == ([2, 3] if inter else [3, 11])
    assert torch.all(out[~torch.isnan(out)] == 0)


def test_qk_positions_default_to_rows_and_outputs_in_place():
    c = QkCase(torch.float32, 50, 2, 2, 32, 32, "l2")
    q, k = c.q.contiguous(), c.k.contiguous()
    a = gdn.gdn_qk_norm_rope(q, k, c.cos, c.sin, norm="l2")
    b = gdn.gdn_qk_norm_rope(q, k, c.cos, c.sin, positions=torch.arange(50, dtype=torch.int32, device=DEV), norm="l2")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    gdn.gdn_qk_norm_rope(q, k, c.cos, c.sin, norm="l2", q_out=q, k_out=k)
    assert torch.equal(a[0], q) and torch.equal(a[1], k)
    wide = torch.zeros(50, 200, device=DEV)
    dq, dk = wide[:, :64].unflatten(1, (2, 32)), wide[:, 68:132].unflatten(1, (2, 32))
    g = gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, norm="l2")
    gdn.gdn_qk_norm_rope_bwd(c.q, c.k, c.cos, c.sin, c.dq, c.dk, norm="l2", dq=dq, dk=dk)
    assert torch.equal(dq, g["dq"]) and torch.equal(dk, g["dk"])
    assert torch.all(wide[:, 64:68] == 0) and torch.all(wide[:, 132:] == 0)
    none = torch.empty(0, 2, 32, device=DEV)
    qo, _ = gdn.gdn_qk_norm_rope(none, none, c.cos, c.sin)
    w = torch.ones(32, device=DEV)
    g = gdn.gdn_qk_norm_rope_bwd(none, none, c.cos, c.sin, none, none, q_weight=w, k_weight=w)
    assert qo.shape == (0, 2, 32) and torch.all(g["dq_weight"] == 0) and torch.all(g["dk_weight"] == 0)


# ---------------------------------------------------------------- offsets past 2^31 values

def test_offsets_past_32_bits():
    """A batch whose last sequence lies behind 2^31 values: its bits alone and in place, for the
    conv's gradient, the q/k norm and its gradient, and the scan with its gradient."""
    C, L, tail = 8192, 262300, 70
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    T = L + tail
    assert L * C > 2 ** 31

    def big(width):
        t = torch.zeros(T, width, dtype=torch.bfloat16, device=DEV)
        t[L:] = rn(tail, width).to(torch.bfloat16)
        return t

    cu = torch.tensor([0, L, T], dtype=torch.int32, device=DEV)
    one = torch.tensor([0, tail], dtype=torch.int32, device=DEV)
    x, dy = big(C), big(C)
    w = rn(C, 4)
    g, a = gdn.gdn_causal_conv1d_bwd(x, w, cu, dy), gdn.gdn_causal_conv1d_bwd(x[L:], w, one, dy[L:])
    assert torch.equal(bits(g["dx"][L:]), bits(a["dx"])) and torch.all(g["dx"][:L - 3] == 0)
    del g, a
    q = x.unflatten(1, (64, 128))
    th = rn(97, 64)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) % 97
    kw = dict(cos=th.cos(), sin=th.sin())
    big_q, _ = gdn.gdn_qk_norm_rope(q, q[:, :1], positions=pos, **kw)
    sub_q, _ = gdn.gdn_qk_norm_rope(q[L:], q[L:, :1], positions=pos[L:], **kw)
    assert torch.equal(bits(big_q[L:]), bits(sub_q)) and torch.all(big_q[:L] == 0)
    del big_q, sub_q
    d = dy.unflatten(1, (64, 128))
    big_g = gdn.gdn_qk_norm_rope_bwd(q, q[:, :1], d_q_out=d, d_k_out=d[:, :1].contiguous(), positions=pos, **kw)
    sub_g = gdn.gdn_qk_norm_rope_bwd(q[L:], q[L:, :1], d_q_out=d[L:], d_k_out=d[L:, :1].contiguous(), positions=pos[L:], **kw)
    assert torch.equal(bits(big_g["dq"][L:]), bits(sub_g["dq"])) and torch.equal(bits(big_g["dk"][L:]), bits(sub_g["dk"]))
    del big_g, sub_g
    B = big(8).unflatten(1, (1, 8))
    args = lambda s: dict(x=x[s], dt=dy[s], A_log=A_log, B=B[s], C=B[s], dt_bias=bias)  # noqa: E731
    A_log, bias = rn(C, 8) * 0.2, rn(C) - 3
    whole, last = slice(None), slice(L, T)
    y, ya = gdn.gdn_selective_scan_fwd(cu_seqlens=cu, **args(whole)), gdn.gdn_selective_scan_fwd(cu_seqlens=one, **args(last))
    assert torch.equal(bits(y[L:]), bits(ya))
    del y, ya
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=cu, d_out=dy, need_d_init_state=False, **args(whole))
    a = gdn.gdn_selective_scan_bwd(cu_seqlens=one, d_out=dy[L:], need_d_init_state=False, **args(last))
    # the segments differ between the two batches: the last sequence's rows agree up to their rounding
    # and the difference of the segments' decays (a product of at most 128 steps: 128 * 4 u), in the row's largest value
    for k in ("dx", "ddt", "dB", "dC"):
        p, q_ = to_np(g[k][L:]).reshape(tail, -1), to_np(a[k]).reshape(tail, -1)
        assert np.all(np.abs(p - q_) <= 2 * BF16_ROUND * np.abs(q_) + 2e-4 * np.abs(q_).max(1, keepdims=True)), k


# ---------------------------------------------------------------- together

def test_conv_norm_rotation_recurrence_and_back():
    """Conv output, split, normed and rotated into the recurrence, and the gradients back through
    all three, against the same chain of oracles (fp32; the recurrence's bars 2e-3 and 1e-2)."""
    import oracle
    lens, HK, HV, dk, dv, W = [40, 3, 21], 2, 4, 32, 16, 4
    T, C = sum(lens), 2 * HK * dk + HV * dv
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    gen = torch.Generator().manual_seed(21)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, w, b = rn(T, C), rn(C, W) / 2, 0.1 * rn(C)
    th = rn(64, 8)
    cos, sin = th.cos(), th.sin()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    g, beta, do = -torch.rand(T, HV, generator=gen), torch.rand(T, HV, generator=gen), rn(T, HV, dv)
    D = lambda t: t.to(DEV)  # noqa: E731
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y = gdn.gdn_causal_conv1d_fwd(D(x), D(w), cud, bias=D(b))
    heads = lambda t, a, H, d: t[:, a:a + H * d].unflatten(1, (H, d))  # noqa: E731
    q, k, v = heads(y, 0, HK, dk), heads(y, HK * dk, HK, dk), heads(y, 2 * HK * dk, HV, dv).contiguous()
    qn, kn = gdn.gdn_qk_norm_rope(q, k, D(cos), D(sin), positions=D(pos), norm="l2")
    out, _ = gdn.gdn_recurrent_fwd(qn, kn, v, D(g), D(beta), cud, use_qk_l2norm=False)
    r = gdn.gdn_chunk_bwd(qn, kn, v, D(g), D(beta), cud, D(do), use_qk_l2norm=False)
    dyc = torch.empty(T, C, device=DEV)
    gdn.gdn_qk_norm_rope_bwd(q, k, D(cos), D(sin), r["dq"], r["dk"], positions=D(pos), norm="l2", dq=heads(dyc, 0, HK, dk),
                             dk=heads(dyc, HK * dk, HK, dk))
    heads(dyc, 2 * HK * dk, HV, dv).copy_(r["dv"])
    back = gdn.gdn_causal_conv1d_bwd(D(x), D(w), cud, dyc, bias=D(b))
    # the oracles
    yr, _ = ref.causal_conv1d(x, w, cu, bias=b)
    qr, kr, vr = (heads(torch.from_numpy(yr), a, H, d) for a, H, d in ((0, HK, dk), (HK * dk, HK, dk), (2 * HK * dk, HV, dv)))
    cs, sn = cos[pos.long()], sin[pos.long()]
    qnr, knr = (torch.from_numpy(ref.norm_rope(t, None, cs, sn, norm="l2")) for t in (qr, kr))
    f = lambda t: t.float().contiguous()  # noqa: E731
    cut = torch.tensor(cu, dtype=torch.int32)
    outr, _ = oracle.gdn_fwd(f(qnr), f(knr), f(vr), g, beta, cut, use_qk_l2norm=False)
    rr = oracle.gdn_bwd(f(qnr), f(knr), f(vr), g, beta, cut, do, use_qk_l2norm=False)
    dyr = np.concatenate([ref.norm_rope_bwd(t, None, cs, sn, rr[n], norm="l2")[0].reshape(T, -1) for t, n in ((qr, "dq"), (kr, "dk"))] +
                         [np.asarray(rr["dv"], dtype=np.float64).reshape(T, -1)], axis=1)
    br = ref.causal_conv1d_bwd(x, w, cu, dyr, bias=b)
    err = lambda a, c: np.abs(to_np(a) - c).max() / np.abs(c).max()  # noqa: E731
    assert err(out, np.asarray(outr)) < 2e-3
    for n in ("dx", "dweight", "dbias"):
        assert err(back[n], br[n]) < 1e-2, n


def test_conv_then_scan_prompt_and_single_tokens():
    """A prompt through conv and scan, then its last tokens one by one on the same two pools: the bits of one prompt."""
    C, S, W, L, P = 64, 16, 4, 45, 38
    gen = torch.Generator().manual_seed(22)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, z, dt = (rn(L, C).to(torch.bfloat16).to(DEV) for _ in range(3))
    B, Cm = (rn(L, 1, S).to(torch.bfloat16).to(DEV) for _ in range(2))
    w, A_log, D, bias = rn(C, W).to(DEV), rn(C, S).to(DEV), rn(C).to(DEV), (rn(C) - 3).to(DEV)
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)
    fresh = torch.zeros(1, dtype=torch.int32, device=DEV)

    def prompt(n):
        conv, st = torch.randn(2, W - 1, C, device=DEV).to(torch.bfloat16), torch.randn(2, C, S, device=DEV)
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        xc = gdn.gdn_causal_conv1d_fwd(x[:n], w, cu, conv_state=conv, state_indices=slot, has_initial_state=fresh)
        y = gdn.gdn_selective_scan_fwd(xc, dt[:n], A_log, B[:n], Cm[:n], cu, D=D, z=z[:n], dt_bias=bias, state=st, state_indices=slot,
                                       has_initial_state=fresh)
        return y, conv, st

    whole, conv_w, st_w = prompt(L)
    y, conv, st = prompt(P)
    rows = [y]
    for t in range(P, L):
        s = slice(t, t + 1)
        xc = gdn.gdn_causal_conv1d_update(x[s], w, conv, state_indices=slot)
        rows.append(gdn.gdn_selective_scan_update(xc, dt[s], A_log, B[s], Cm[s], st, state_indices=slot, D=D, z=z[s], dt_bias=bias))
    assert torch.equal(bits(torch.cat(rows)), bits(whole))
    assert torch.equal(bits(conv[1]), bits(conv_w[1])) and torch.equal(bits(st[1]), bits(st_w[1]))
