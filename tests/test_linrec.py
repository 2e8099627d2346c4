"""GPU parity, invariance and gradients of the gated linear recurrence against the fp64 oracle
(oracle/linrec_ops.py).

Tolerances, in units of u = 2^-24 of the sum of the terms' magnitudes (the oracle with
magnitude=True).  With g the largest |gate|: sigmoid(g) = 1 / (1 + 2^(-g log2 e)) carries the
exponent's two roundings (2 g u), the hardware exponential (2^-22.5: 3 u), a sum (u) and the
hardware reciprocal (2 u), or two gates' common one with two products more: (2 g + 9) u; 1 - sigmoid one more.
K = decay softplus(a_param) is good to 8 u, so w = K r to E_w = (2 g + 18) u, and m = 1 - e^-w to E_w + 5 u.  log a is off by w E_w + 5 u a
token (its rounding, up to 1.65 u, and m's own 4 u m / a; above w = 1/2 the hardware
exponential, 3 u + 2 w u); over a sequence's L tokens by (2 g + 20) u min(40, s) + 5 u L, s = sum of w
(past s = 40 a term is below e^-40 of itself).  Without an a_param a = sigmoid(g): its error,
e / (1 + e) (2 |g| + 3) u + 6 u, is at most (2 w + 10) u, since |g| <= w for g < 0 and e |g| / (1 + e) < 0.28
for g > 0.  s_t = sqrt(m + m a) is good to (2 g + 28) u, x sigmoid(x_gate) to (2 g + 10) u; with L
roundings of the walk:
    E = 40 + 4 g + 11 L + (2 g + 20) min(40, s).
act(z) adds (8 + 6 max |inner(z)|) u of the result (inner: its sigmoid's argument, 4 roundings).
A gradient multiplies two such recurrences and the factors of a third, 3 E and three times act's share;
da_param's sum adds T, its factor 12 u.  dz's slope p + z p (1 - p) inner'(z) is a sum that cancels: the oracle's
magnitude takes its terms' absolute values, each good to twice act's share.
1 - a below 2^-126, fp32's smallest normal number, counts as 0 (a gate of 100 without a_param): sqrt(1 - a^2)
is off by up to 2^-62.5 there, its slope's product m a^2 / s by 2^-63.5, whatever the token multiplies it with, and h by the sum over
L tokens.  Where a batch has such tokens, this floor is added.
A bf16 output adds its own rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from oracle import linrec_ops as ref
from helpers import BF16_ROUND, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
INF = float("inf")
BF, F32 = torch.bfloat16, torch.float32
LENS = [33, 0, 1, 70, 16, 2, 64, 31]


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


class Case:
    """Inputs of a ragged batch; x, the gates and z as columns of wider rows when strided."""

    def __init__(self, lens, C, dtype, seed, param=True, xgate=True, act="", scale="sqrt", strided=False, behind=0):
        gen = torch.Generator().manual_seed(seed)
        T = sum(lens) + behind

        def rows(shift=0.0, by=1.0):
            v = torch.randn(T, C + (24 if strided else 0), generator=gen) * by + shift
            v = v.to(dtype).to(DEV)
            return v[:, 8:-16] if strided else v

        self.lens, self.C, self.dtype = lens, C, dtype
        self.cu_list = np.concatenate([[0], np.cumsum(lens)]).tolist()
        self.cu = torch.tensor(self.cu_list, dtype=torch.int32, device=DEV)
        self.x, self.ag = rows(), rows() if param else rows(2.0, 1.5)
        self.xg, self.z = rows() if xgate else None, rows() if act else None
        keep = 0.9 + 0.099 * torch.rand(C, generator=gen)
        keep[::5] = 0.02  # some that forget at once
        self.ap = torch.log(torch.expm1(-torch.log(keep) / 8)).to(DEV) if param else None
        self.dy = torch.randn(T, C, generator=gen).to(dtype).to(DEV)
        self.h0, self.gT = (torch.randn(len(lens), C, generator=gen).to(DEV) for _ in range(2))
        self.kw = dict(input_scale=scale, activation=act or "silu")

    def args(self, t=slice(None)):
        return dict(x=self.x[t], a_gate=self.ag[t], a_param=self.ap, x_gate=None if self.xg is None else self.xg[t],
                    z=None if self.z is None else self.z[t], **self.kw)

    def units(self):
        """E, act's share, and the floor."""
        ag = to_np(self.ag)[:self.cu_list[-1]]
        ag = ag[np.isfinite(ag)]
        g = max(np.abs(ag).max(initial=0), 0 if self.xg is None else np.abs(to_np(self.xg)).max(initial=0))
        w = ref.exponents(np.nan_to_num(to_np(self.ag), nan=0, posinf=700, neginf=-700), None if self.ap is None else to_np(self.ap), 8.0)
        s = max(w[a:b].sum(0).max() for a, b in zip(self.cu_list, self.cu_list[1:]))
        share = 0.0 if self.z is None else 8 + 6 * np.abs(ref.inner(self.kw["activation"], to_np(self.z))).max(initial=0)
        floor = 1e-30
        if self.kw["input_scale"] == "sqrt" and (w < 2.0 ** -126).any():
            G = ref.linear_recurrence_bwd(cu=self.cu_list, d_out=self.dy, d_final_state=self.gT, magnitude=True, **dict(self.args(), x_gate=None, input_scale="one"))["dx"]
            f = 1 if self.z is None else 1 + np.abs(to_np(self.z)).max()
            floor = 2.0 ** -62 * max(self.lens) * (1 + np.nanmax(G)) * (1 + np.nanmax(np.abs(to_np(self.x)))) * f
        return 40 + 4 * g + 11 * max(self.lens) + (2 * g + 20) * min(40.0, s), share, floor


def check(got, want, mag, units, dtype, floor=1e-30):
    got = to_np(got)
    ok = ~np.isnan(want)
    bound = units * U * mag[ok] + (BF16_ROUND if dtype == BF else U) * np.abs(want[ok]) + floor
    err = np.abs(got[ok] - want[ok])
    assert np.all(err <= bound), (err / bound).max()


def check_forward(c, y, pool, init, rows=slice(None)):
    want, fin = ref.linear_recurrence(cu=c.cu_list, init_state=init, **c.args())
    mag, fmag = ref.linear_recurrence(cu=c.cu_list, init_state=init, magnitude=True, **c.args())
    E, share, floor = c.units()
    check(y, want, mag, E + share, c.dtype, floor)
    if pool is not None:
        check(pool[rows], fin, fmag, E, F32, floor)


def check_backward(c, states=True, **kw):
    st = dict(init_state=c.h0, d_final_state=c.gT) if states else {}
    g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, need_d_init_state=states, **st, **kw, **c.args())
    want = ref.linear_recurrence_bwd(cu=c.cu_list, d_out=c.dy, **st, **c.args())
    mag = ref.linear_recurrence_bwd(cu=c.cu_list, d_out=c.dy, magnitude=True, **st, **c.args())
    E, share, floor = c.units()
    for k in ("dx", "da_gate") + (("dx_gate",) if c.xg is not None else ()) + (("dz",) if c.z is not None else ()) + \
            (("da_param",) if c.ap is not None else ()) + (("d_init_state",) if states else ()):
        wide = k in ("da_param", "d_init_state")
        assert g[k].dtype == (F32 if wide else c.dtype)
        check(g[k], want[k], mag[k], 3 * E + 3 * share + (sum(c.lens) + 12 if k == "da_param" else 0), F32 if wide else c.dtype, floor)
    for k, t in (("dx_gate", c.xg), ("dz", c.z), ("da_param", c.ap)):
        assert (g[k] is None) == (t is None)
    assert (g["d_init_state"] is None) == (not states)
    return g


# C: one, two and many blocks of channels, whole and in part; every scale, activation, gate and type
GRID = [(BF, 200, True, True, "gelu", "sqrt"), (F32, 72, True, True, "", "sqrt"), (F32, 140, False, False, "silu", "linear"), (BF, 8, True, False, "silu", "one"),
        (F32, 4, False, True, "gelu", "sqrt"), (BF, 64, False, False, "", "linear"), (BF, 1040, True, True, "", "linear"), (F32, 516, True, False, "gelu", "one")]


@pytest.mark.parametrize("dtype,C,param,xgate,act,scale", GRID)
@pytest.mark.parametrize("strided", [False, True])
def test_forward_vs_oracle(dtype, C, param, xgate, act, scale, strided):
    c = Case(LENS, C, dtype, 11, param, xgate, act, scale, strided=strided, behind=3)
    N = len(LENS)
    pool0 = torch.randn(N + 4, C, generator=torch.Generator().manual_seed(1)).to(DEV)
    slots = torch.randperm(N + 4, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
    has = torch.tensor([1, 1, 0, 1, 0, 1, 1, 0], dtype=torch.int32)
    pool, out = pool0.clone(), torch.full((sum(LENS) + 3, C), float("nan"), dtype=dtype, device=DEV)
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, state_indices=slots.to(DEV), has_initial_state=has.to(DEV), out=out, **c.args())
    assert y is out
    check_forward(c, y, pool, to_np(pool0)[slots.long().numpy()] * has.numpy()[:, None], slots.long())
    spare = sorted(set(range(N + 4)) - set(slots.tolist()))
    assert torch.equal(bits(pool[spare]), bits(pool0[spare]))


@pytest.mark.parametrize("dtype,C,param,xgate,act,scale", GRID)
def test_bits_do_not_depend_on_the_batch_or_on_how_tokens_arrive(dtype, C, param, xgate, act, scale):
    lens = [77, 5, 230, 1]
    c = Case(lens, C, dtype, 12, param, xgate, act, scale)
    pool = c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    one = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    for n in (0, 2):  # alone
        t = slice(c.cu_list[n], c.cu_list[n + 1])
        st = c.h0[n:n + 1].clone()
        alone = gdn.gdn_linear_recurrence_fwd(cu_seqlens=one(lens[n]), state=st, **c.args(t))
        assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(st[0]), bits(pool[n]))
    # in chained calls, the last tokens one by one beside another sequence
    a = c.cu_list[2]
    st = torch.zeros(3, C, device=DEV)
    st[2] = c.h0[2]
    idx = torch.tensor([2], dtype=torch.int32, device=DEV)
    parts = [gdn.gdn_linear_recurrence_fwd(cu_seqlens=one(m - k), state=st, state_indices=idx, **c.args(slice(a + k, a + m)))
             for k, m in ((0, 33), (33, 34), (34, 220))]
    two = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    for t in range(220, 230):
        parts.append(gdn.gdn_linear_recurrence_update(state=st, state_indices=two, **c.args(torch.tensor([a + t, t], device=DEV)))[:1])
    assert torch.equal(bits(torch.cat(parts)), bits(y[a:a + 230])) and torch.equal(bits(st[2]), bits(pool[2]))


@pytest.mark.parametrize("dtype,N,C,longest", [(BF, 110, 2056, 130), (F32, 110, 1036, 130), (BF, 3, 4104, 700), (F32, 2, 8200, 300), (BF, 700, 40, 9), (BF, 9, 264, 1500), (F32, 5, 4100, 200)])
def test_large_batches_agree_with_a_sequence_alone(dtype, N, C, longest):
    lens = [(37 * i) % longest + (longest // 2 if i == 0 else 0) for i in range(N)]
    c = Case(lens, C, dtype, 13, act="gelu")
    pool = c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    for n in range(0, N, max(1, N // 40)):
        t = slice(c.cu_list[n], c.cu_list[n + 1])
        st = c.h0[n:n + 1].clone()
        alone = gdn.gdn_linear_recurrence_fwd(cu_seqlens=torch.tensor([0, lens[n]], dtype=torch.int32, device=DEV), state=st, **c.args(t))
        assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(st[0]), bits(pool[n])), n


@pytest.mark.parametrize("dtype,C,lens", [(BF, 24, [521, 2, 259]), (F32, 20, [263, 0, 130, 5]), (BF, 1032, [258]), (F32, 36, [1, 2, 3])])
def test_few_channels_walk_as_single_tokens_do(dtype, C, lens):
    """Batches of few CTAs, a half of a warp for each: whole and part tiles, units and channel blocks."""
    c = Case(lens, C, dtype, 27, act="silu")
    pool, st = c.h0.clone(), c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    for n, (lo, hi) in enumerate(zip(c.cu_list, c.cu_list[1:])):
        slot = torch.tensor([n], dtype=torch.int32, device=DEV)
        one = [gdn.gdn_linear_recurrence_update(state=st, state_indices=slot, **c.args(slice(t, t + 1))) for t in range(lo, hi)]
        assert not one or torch.equal(bits(torch.cat(one)), bits(y[lo:hi])), n
    assert torch.equal(bits(st), bits(pool))


@pytest.mark.parametrize("dtype,B,C", [(BF, 300, 4160), (F32, 150, 4164), (F32, 37, 1000), (BF, 1, 8)])
@pytest.mark.parametrize("param,act", [(True, "gelu"), (False, "silu"), (True, "")])
def test_large_updates_agree_with_prompts_of_one_token(dtype, B, C, param, act):
    c = Case([1] * B, C, dtype, 24, param=param, act=act, strided=True)
    a, b = c.h0.clone(), c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=a, **c.args())
    z = gdn.gdn_linear_recurrence_update(state=b, **c.args())
    assert torch.equal(bits(y), bits(z)) and torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("param,xgate,scale", [(True, True, "sqrt"), (False, False, "linear"), (True, False, "one")])
@pytest.mark.parametrize("dtype,N,C,every", [(BF, 300, 264, 135), (F32, 300, 260, 135), (BF, 5000, 64, 608), (F32, 40, 9000, 3), (BF, 1, 9800, 1)])
def test_short_sequences_with_long_ones_among_them(dtype, N, C, every, param, xgate, scale):
    """Lengths around 32, empty ones, and long ones `every` sequences apart."""
    lens = [[1, 0, 32, 33, 7, 1, 31, 2][(5 * i) % 8] for i in range(N)]
    lens[5 % N::every] = [(40 + 97 * i) % 700 if N < 5000 else 300 for i in range(len(lens[5 % N::every]))] if N > 40 else [60] * len(lens[5 % N::every])
    c = Case(lens, C, dtype, 26, param, xgate, "gelu", scale, strided=True, behind=9)
    idx = torch.randperm(N + 2, generator=torch.Generator().manual_seed(4))[:N].to(torch.int32)
    idx[3::11] = -1
    has = (torch.arange(N) % 3 != 0).to(torch.int32).to(DEV)
    pool0 = torch.randn(N + 2, C, generator=torch.Generator().manual_seed(5)).to(DEV)
    pool, out = pool0.clone(), torch.full((sum(lens) + 9, C), 7.0, dtype=dtype, device=DEV)
    gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, state_indices=idx.to(DEV), has_initial_state=has, out=out, **c.args())
    assert torch.all(out[sum(lens):] == 7)
    for n in {*range(0, N, max(1, N // 40)), *range(5 % N, N, max(every, N // 20)), 3 % N}:
        t, slot = slice(c.cu_list[n], c.cu_list[n + 1]), int(idx[n])
        st = pool0[slot:slot + 1].clone() if slot >= 0 and has[n] else torch.zeros(1, C, device=DEV)
        y = []
        for k in range(t.start, t.stop, 257):  # alone, in chained calls
            part = slice(k, min(k + 257, t.stop))
            y.append(gdn.gdn_linear_recurrence_fwd(cu_seqlens=torch.tensor([0, part.stop - k], dtype=torch.int32, device=DEV), state=st, **c.args(part)))
        if y:
            assert torch.equal(bits(torch.cat(y)), bits(out[t])), n
        if slot >= 0:
            assert torch.equal(bits(st[0]), bits(pool[slot])), n
    spare = sorted(set(range(N + 2)) - set(idx.tolist()))
    assert torch.equal(bits(pool[spare]), bits(pool0[spare]))


@pytest.mark.parametrize("dtype,C,longest", [(BF, 264, 5003), (F32, 132, 5003), (BF, 1040, 40001), (F32, 516, 20001)])
@pytest.mark.parametrize("where", [0, 100, 299])
def test_a_long_prompt_among_single_tokens(dtype, C, longest, where):
    """Decoding sequences of one token and a prompt of thousands in one batch, by either form that their mean length takes: the single
    tokens have an update's bits, the prompt those it has alone, and the gradient holds at both."""
    lens = [1] * 300
    lens[where] = longest
    c = Case(lens, C, dtype, 42, act="gelu")
    pool, st = c.h0.clone(), c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    t, single = slice(where, where + longest), [n for n in range(300) if n != where]
    rows = torch.tensor([c.cu_list[n] for n in single], device=DEV)
    alone = gdn.gdn_linear_recurrence_fwd(cu_seqlens=torch.tensor([0, longest], dtype=torch.int32, device=DEV), state=st[where:where + 1], **c.args(t))
    one = gdn.gdn_linear_recurrence_update(state=st, state_indices=torch.tensor(single, dtype=torch.int32, device=DEV), **c.args(rows))
    assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(one), bits(y[rows])) and torch.equal(bits(st), bits(pool))
    if longest < 10000:
        check_forward(c, y, pool, c.h0)
        check_backward(c)


@pytest.mark.parametrize("dtype,B,C", [(BF, 1001, 4160), (BF, 250, 8200), (F32, 1001, 4164)])
def test_large_updates_skip_rows_anywhere(dtype, B, C):
    """Threads that take several rows, with skipped ones first, last and side by side among them."""
    c = Case([1] * B, C, dtype, 25, act="gelu")
    slots = torch.randperm(B, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    slots[::3] = -1
    slots[7:40] = B
    idx, keep = slots.to(DEV), (slots >= 0) & (slots < B)
    a, b = c.h0.clone(), c.h0.clone()
    out = torch.full((B, C), 7.0, dtype=dtype, device=DEV)
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=a, state_indices=idx, **c.args())
    gdn.gdn_linear_recurrence_update(state=b, state_indices=idx, out=out, **c.args())
    keep = keep.to(DEV)
    assert torch.equal(bits(out[keep]), bits(y[keep])) and torch.all(out[~keep] == 7) and torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("dtype,C,param,xgate,act,scale", GRID)
def test_update_vs_oracle_and_skips(dtype, C, param, xgate, act, scale):
    B = 11
    c = Case([1] * B, C, dtype, 14, param, xgate, act, scale, strided=True)
    idx = torch.tensor([3, -1, 0, 12, 7, 13, 5, 1, 2, 9, 4], dtype=torch.int32, device=DEV)  # -1 and 13: skipped
    pool0 = torch.randn(13, C, device=DEV)
    pool, out = pool0.clone(), torch.full((B, C), 7.0, dtype=dtype, device=DEV)
    gdn.gdn_linear_recurrence_update(state=pool, state_indices=idx, out=out, **c.args())
    keep = [i for i in range(B) if 0 <= int(idx[i]) < 13]
    slot = idx[keep].long()
    cu, rows = list(range(len(keep) + 1)), torch.tensor(keep, device=DEV)
    want, fin = ref.linear_recurrence(cu=cu, init_state=pool0[slot], **c.args(rows))
    mag, fmag = ref.linear_recurrence(cu=cu, init_state=pool0[slot], magnitude=True, **c.args(rows))
    E, share, floor = c.units()
    check(out[keep], want, mag, E + share, dtype, floor)
    check(pool[slot], fin, fmag, E, F32, floor)
    assert torch.all(out[[i for i in range(B) if i not in keep]] == 7)
    spare = sorted(set(range(13)) - set(slot.tolist()))
    assert torch.equal(bits(pool[spare]), bits(pool0[spare]))


@pytest.mark.parametrize("dtype,C,param,xgate,act,scale", GRID)
@pytest.mark.parametrize("states", [False, True])
def test_backward_vs_oracle(dtype, C, param, xgate, act, scale, states):
    check_backward(Case(LENS, C, dtype, 17, param, xgate, act, scale, strided=states), states)


@pytest.mark.parametrize("dtype,C,lens", [(BF, 264, [700, 0, 1, 130, 128, 127]), (F32, 36, [1500]), (BF, 8, [1, 2, 0, 3000]), (F32, 516, [(13, 0, 64, 1, 40)[i % 5] for i in range(200)]),
                                          (BF, 2056, [65, 300, 129])])
@pytest.mark.parametrize("param,act", [(True, "gelu"), (False, "")])
def test_backward_of_sequences_of_every_length(dtype, C, lens, param, act):
    """Also: a workspace filled with NaN changes nothing, and the bits repeat."""
    c = Case(lens, C, dtype, 38, param, param, act, "sqrt" if param else "linear")
    g = check_backward(c)
    shape = gdn.LinrecShape(len(lens), sum(lens), C, int(dtype == BF), 0, 0, 8.0, C, C, C, C)
    ws = torch.full((gdn.lib().gdn_linear_recurrence_bwd_workspace_size(shape),), 255, dtype=torch.uint8, device=DEV)
    again = check_backward(c, workspace=ws)
    for k in g:
        assert g[k] is None or torch.equal(bits(g[k]), bits(again[k])), k
    with pytest.raises(gdn.GdnError):
        check_backward(c, workspace=ws[:8])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_sequences_than_a_grids_second_dimension_holds(dtype):
    lens = [(1, 0, 2, 1)[i % 4] for i in range(66000)]
    lens[40000] = 300
    c = Case(lens, 8, dtype, 41, act="silu")
    pool = c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    check_forward(c, y, pool, c.h0)
    check_backward(c)


def test_gradient_by_differences():
    """The kernels' gradient against differences of the kernels' forward, fp32."""
    c = Case([5, 3], 8, F32, 51, act="gelu")
    # step 1/64: the differences' own error is of third order, 2e-4 of values of order one, the forward's 1e-6 over the step 1e-4
    loss = lambda a, h0: float((gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=h0, **a).double() * c.dy.double()).sum() + (h0.double() * c.gT.double()).sum())  # noqa: E731
    g = check_backward(c)
    for k, name in (("x", "dx"), ("a_gate", "da_gate"), ("x_gate", "dx_gate"), ("z", "dz"), ("a_param", "da_param")):
        for at in ((0, 1), (4, 5), (7, 6)):
            at = at[1:] if k == "a_param" else at
            v = []
            for s in (1, -1):
                a = dict(c.args())
                a[k] = a[k].clone()
                a[k][at] += s / 64
                v.append(loss(a, c.h0.clone()))
            assert abs((v[0] - v[1]) * 32 - float(g[name][at])) < 2e-3, (k, at)


# ---------------------------------------------------------------- values at the edges

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", ["sqrt", "linear"])
def test_gates_far_out(dtype, scale):
    """Under an a_param a gate of -inf keeps the state's bits and has no gradient; without one it forgets.  An a_param past
    fp32's range forgets at once unless the gate is shut."""
    c = Case([33, 5, 0, 18], 24, dtype, 31, act="silu", scale=scale)
    c.ag[::3] = -INF
    c.ag[1::9] = INF
    pool = c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    check_forward(c, y, pool, c.h0)
    g = check_backward(c)
    assert torch.all(g["da_gate"][:56:3] == 0)
    shut = dict(c.args(), a_gate=torch.full_like(c.ag, -INF))
    for ap in (c.ap, torch.full_like(c.ap, 3e38)):
        pool = c.h0.clone()
        gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **dict(shut, a_param=ap))
        assert torch.equal(bits(pool), bits(c.h0))
    d = Case([33, 5, 0, 18], 24, dtype, 32, param=False, scale=scale)
    d.ag[::4] = -INF
    d.ag[1::9] = 100.0
    d.ag[2::9] = -100.0
    pool = d.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=d.cu, state=pool, **d.args())
    check_forward(d, y, pool, d.h0)
    check_backward(d)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", ["sqrt", "linear"])
def test_exponents_around_a_quarter_have_one_form(dtype, scale):
    """K = decay softplus(a_param) just below and above 1/4, where 1 - e^-w goes from one form to the other, beside channels far past
    it: which channels share a thread differs between a prompt and single tokens, the bits do not."""
    C, T = 2048, 192
    # softplus(0) = log 2; from -1e-6 to 1e-6 it takes every fp32 value there, K some ulp each
    ap = torch.linspace(-1e-6, 1e-6, C, device=DEV)
    ap[::8], ap[5::16] = 8.0, 8.0
    gen = torch.Generator().manual_seed(28)
    x, xg = (torch.randn(T, C, generator=gen).mul(4).to(dtype).to(DEV) for _ in range(2))
    ag = torch.full((T, C), 30.0, dtype=dtype, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for k in range(-2, 3):  # decays a few ulp apart
        kw = dict(a_param=ap, input_scale=scale, decay=float(np.float32(0.25 / np.log(2)) * (1 + k * 2.0 ** -23)))
        a, b = torch.zeros(1, C, device=DEV), torch.zeros(1, C, device=DEV)
        y = gdn.gdn_linear_recurrence_fwd(x, ag, cu, x_gate=xg, state=a, **kw)
        z = torch.cat([gdn.gdn_linear_recurrence_update(x[t:t + 1], ag[t:t + 1], b, x_gate=xg[t:t + 1], **kw) for t in range(T)])
        assert torch.equal(bits(y), bits(z)) and torch.equal(bits(a), bits(b)), k


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", ["sqrt", "linear"])
@pytest.mark.parametrize("xgate", [True, False])
def test_open_forget_gates_keep_the_state(dtype, scale, xgate):
    """Without an a_param a gate of +inf, or of 30 and nothing taken in, keeps the state's bits whatever x_gate is, and the
    gradient's; no gate makes it grow.  Gates of 12: a state of 1 stays within [0.97, 1], where a token's two roundings, of a = 1 - 6e-6
    and of the product, are half of u = 2^-24 each."""
    C, T = 1024, 4096
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    x = torch.zeros(T, C, dtype=dtype, device=DEV)
    xg = torch.linspace(-12, 12, C, device=DEV).to(dtype).expand(T, C).contiguous() if xgate else None
    one = torch.ones(1, C, device=DEV)

    def run(gate, state, x=x):
        ag = torch.full((T, C), gate, dtype=dtype, device=DEV)
        y = gdn.gdn_linear_recurrence_fwd(x, ag, cu, x_gate=xg, state=state, input_scale=scale)
        return y, gdn.gdn_linear_recurrence_bwd(x, ag, cu, torch.zeros_like(x), x_gate=xg, init_state=one, d_final_state=one, input_scale=scale)["d_init_state"]

    for gate in (INF, 100.0, 30.0):
        st = one.clone()
        y, d_init = run(gate, st, torch.randn(T, C, device=DEV).to(dtype) if gate == INF else x)
        assert torch.equal(st, one) and torch.all(y == 1) and torch.equal(d_init, one), gate
        st, ag = one.clone(), torch.full((1, C), gate, dtype=dtype, device=DEV)
        for _ in range(3):
            gdn.gdn_linear_recurrence_update(x[:1], ag, st, x_gate=None if xg is None else xg[:1], input_scale=scale)
        assert torch.equal(st, one), gate
    for gate in (0.0, 1.0, 4.0, 8.0, 16.0):
        st = one.clone()
        _, d_init = run(gate, st)
        assert torch.all(st <= 1) and torch.all(d_init <= 1), gate
    st = one.clone()
    _, d_init = run(12.0, st)
    want = np.exp(-T * np.logaddexp(0, -12.0))
    assert np.abs(to_np(st) - want).max() < 1.1 * T * U and np.abs(to_np(d_init) - want).max() < 1.1 * T * U


@pytest.mark.parametrize("dtype", [F32, BF])
def test_decays_next_to_one(dtype):
    """1 - a and 1 - a^2 keep their relative accuracy: with K = 8e-6 and less they are past what a's own rounding shows."""
    c = Case([64, 3], 16, dtype, 33)
    c.ap = torch.linspace(-80, -13, 16).to(DEV)
    pool = torch.zeros_like(c.h0)
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    check_forward(c, y, pool, torch.zeros_like(c.h0))
    check_backward(c)
    c.ap = torch.full((16,), -200.0, device=DEV)  # K underflows to 0: nothing is forgotten or taken in, and no gradient is NaN
    pool = c.h0.clone()
    gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    assert torch.equal(bits(pool), bits(c.h0))
    g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, **c.args())
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("ap", [INF, 3e38, 4.25e37, 1e30])
def test_rates_at_the_end_of_the_range(dtype, ap):
    """K = 8 a_param past fp32's range, or near its end: open gates forget at once, with gradients of 0 and none that is NaN, whatever x_gate is."""
    C, T = 4096, 5
    xg = torch.linspace(-12, 12, C, device=DEV).to(dtype).expand(T, C).contiguous()
    x, one = torch.ones(T, C, dtype=dtype, device=DEV), torch.ones(1, C, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for gate in (INF, 30.0, 5.0, 0.0):
        ag = torch.full((T, C), gate, dtype=dtype, device=DEV)
        kw = dict(a_param=torch.full((C,), ap, device=DEV), x_gate=xg)
        st = 3 * one
        y = gdn.gdn_linear_recurrence_fwd(x, ag, cu, state=st, **kw)
        want = torch.sigmoid(xg.double())
        bound = (2 * 12 + 10) * U + (BF16_ROUND if dtype == BF else U)  # x sigmoid(x_gate), s = 1 (module docstring)
        assert torch.all((y.double() - want).abs() <= bound * want)
        g = gdn.gdn_linear_recurrence_bwd(x, ag, cu, x, init_state=one, **kw)
        assert torch.all(g["da_gate"] == 0) and torch.all(g["da_param"] == 0) and torch.all(g["d_init_state"] == 0)
        assert torch.all((g["dx"].double() - want).abs() <= bound * want) and torch.isfinite(g["dx_gate"]).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_branch_values_far_out(act):
    """z up to the type's range: act(z) is z or 0, its slope 1 or 0."""
    z = torch.tensor([-1e30, -1e19, -300.0, -30.0, 30.0, 300.0, 1e19, 1e30], device=DEV).expand(3, 8).contiguous()
    one, ag = torch.ones(3, 8, device=DEV), torch.full((3, 8), -INF, device=DEV)  # a = 0 without a_param: h = x
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    kw = dict(z=z, input_scale="linear", activation=act)
    y = gdn.gdn_linear_recurrence_fwd(one, ag, cu, **kw)
    assert torch.equal(y, z.clamp(min=0)) or torch.allclose(y, z.clamp(min=0), rtol=1e-6, atol=1e-10)
    g = gdn.gdn_linear_recurrence_bwd(one, ag, cu, one, **kw)
    assert torch.allclose(g["dz"], (z > 0).float(), rtol=0, atol=1e-10)


def test_nan_stays_in_its_sequence_and_channel():
    c = Case([40, 9, 50], 72, BF, 34, act="silu")
    pool = c.h0.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    c.x[20, 5] = float("nan")
    p2 = c.h0.clone()
    y2 = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=p2, **c.args())
    g2 = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    assert torch.isnan(y2[20:40, 5]).all() and torch.isnan(p2[0, 5])
    y2[20:40, 5], p2[0, 5] = y[20:40, 5], pool[0, 5]
    assert torch.equal(bits(y2), bits(y)) and torch.equal(bits(p2), bits(pool))
    rest = [i for i in range(72) if i != 5]
    for k in ("dx", "da_gate", "dx_gate", "dz", "d_init_state"):
        assert torch.equal(bits(g2[k][:, rest]), bits(g[k][:, rest])), k
        lo = 1 if k == "d_init_state" else 40
        assert torch.equal(bits(g2[k][lo:]), bits(g[k][lo:])), k
    assert torch.equal(bits(g2["da_param"][rest]), bits(g["da_param"][rest]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("param,scale", [(True, "sqrt"), (False, "linear"), (True, "one")])
@pytest.mark.parametrize("which", ["xg", "ag"])
def test_nan_in_one_gate_leaves_the_other(dtype, param, scale, which):
    """A gate that is not a number reaches what the definition says and nothing else: not the other gate's sigmoid, and so not the
    gradients of the tokens before (x_gate) or behind (a_gate)."""
    lens, at, C = [70, 90, 20], 110, 24
    c = Case(lens, C, dtype, 35, param, act="silu", scale=scale)
    call = lambda: (gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, **c.args()),  # noqa: E731
                    gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args()))
    y0, g0 = call()
    getattr(c, which)[at, 5] = float("nan")
    y, g = call()
    with np.errstate(invalid="ignore"):
        want = ref.linear_recurrence_bwd(cu=c.cu_list, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
        wy, _ = ref.linear_recurrence(cu=c.cu_list, init_state=c.h0, **c.args())
    assert np.array_equal(np.isnan(to_np(y)), np.isnan(wy))
    ok = ~torch.isnan(y)
    assert torch.equal(y[ok], y0[ok])
    for k in ("dx", "da_gate", "dx_gate", "dz", "d_init_state") + (("da_param",) if param else ()):
        nan = np.isnan(want[k])
        assert np.array_equal(np.isnan(to_np(g[k])), nan), k
        if k != "da_param":
            assert nan.any() == (k != "d_init_state" or which == "ag") and not nan.all()
        ok = torch.from_numpy(~nan).to(DEV)
        if which == "ag" and k in ("dx", "dx_gate"):
            ok[at, 5] = False  # dx, dx_gate: p by its own reciprocal here
        assert torch.equal(g[k][ok], g0[k][ok]), k


@pytest.mark.parametrize("dtype", [F32, BF])
def test_nan_in_a_rate_is_seen_in_its_gradient(dtype):
    """A channel whose a_param is not a number: its outputs and gradients, da_param's among them, are none either; the others' bits stay."""
    c = Case([40, 9, 0, 33], 72, dtype, 36, act="silu")
    call = lambda: (gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, **c.args()),  # noqa: E731
                    gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args()))
    y0, g0 = call()
    c.ap[7] = float("nan")
    y, g = call()
    rest = [i for i in range(72) if i != 7]
    assert torch.isnan(y[:, 7]).all() and torch.equal(bits(y[:, rest]), bits(y0[:, rest]))
    assert torch.isnan(g["da_param"][7]) and torch.isnan(g["da_gate"][:, 7]).all()
    for k in g:
        assert torch.equal(bits(g[k][..., rest]), bits(g0[k][..., rest])), k


# ---------------------------------------------------------------- rows, slots, streams, refusals

def test_rows_behind_the_last_sequence_are_neither_read_nor_written():
    c = Case([40, 3], 64, BF, 16, act="gelu", behind=5)
    for t in (c.x, c.ag, c.xg, c.z, c.dy):
        t[43:] = float("nan")
    out = torch.full((48, 64), 3.0, dtype=BF, device=DEV)
    gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, out=out, **c.args())
    assert torch.all(out[43:] == 3) and torch.isfinite(out[:43]).all()
    g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, **c.args())
    for k in ("dx", "da_gate", "dx_gate", "dz"):
        assert torch.isfinite(g[k][:43]).all(), k
    assert torch.isfinite(g["da_param"]).all() and torch.isfinite(g["d_init_state"]).all()


def test_no_tokens_padding_only_and_slots_outside_the_pool():
    x = torch.empty(0, 16, device=DEV)
    st = torch.randn(3, 16, device=DEV)
    s0, cu = st.clone(), torch.zeros(4, dtype=torch.int32, device=DEV)
    has = torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)
    assert gdn.gdn_linear_recurrence_fwd(x, x, cu, state=st, has_initial_state=has).shape == (0, 16)
    assert torch.equal(st[[0, 2]], s0[[0, 2]]) and torch.all(st[1] == 0)
    gT, ap = torch.randn(3, 16, device=DEV), torch.zeros(16, device=DEV)
    g = gdn.gdn_linear_recurrence_bwd(x, x, cu, x, a_param=ap, d_final_state=gT)
    assert torch.equal(g["d_init_state"], gT) and torch.all(g["da_param"] == 0)
    g = gdn.gdn_linear_recurrence_bwd(x, x, cu[:1], x, a_param=ap)
    assert g["d_init_state"].shape == (0, 16) and torch.all(g["da_param"] == 0)
    assert gdn.gdn_linear_recurrence_update(x, x, st).shape == (0, 16)
    c = Case([0, 0], 16, F32, 25, behind=5)
    for t in (c.x, c.ag, c.xg, c.dy):
        t[:] = float("nan")
    st, out = c.h0.clone(), torch.full((5, 16), 3.0, device=DEV)
    gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=st, out=out, **c.args())
    assert torch.all(out == 3) and torch.equal(st, c.h0)
    g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    assert torch.equal(g["d_init_state"], c.gT) and torch.all(g["da_param"] == 0)
    c = Case([9, 4, 6], 16, F32, 26)
    pool = torch.randn(3, 16, device=DEV)
    p0 = pool.clone()
    y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=pool, state_indices=torch.tensor([-1, 3, 1 << 30], dtype=torch.int32, device=DEV), **c.args())
    assert torch.equal(y, gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, **c.args())) and torch.equal(pool, p0)


def test_offsets_past_2_31():
    """Rows so far apart that a token's offset passes 2^31 elements (2 GB and 4 GB of bf16)."""
    T, C, ld = 70, 8, 32 << 20
    wide = torch.zeros(T, ld, dtype=BF, device=DEV)
    c = Case([65, 5], C, BF, 27)
    wide[:, :C], wide[:, 16:16 + C] = c.x, c.ag
    far = dict(c.args(), x=wide[:, :C], a_gate=wide[:, 16:16 + C])
    assert (T - 1) * ld > 2 ** 31
    assert torch.equal(bits(gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, **far)), bits(gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, **c.args())))
    a, b = (gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, **v) for v in (far, c.args()))
    for k in a:
        assert a[k] is None or torch.equal(bits(a[k]), bits(b[k])), k
    s, t = torch.zeros(T, C, device=DEV), torch.zeros(T, C, device=DEV)
    u, v = gdn.gdn_linear_recurrence_update(state=s, **far), gdn.gdn_linear_recurrence_update(state=t, **c.args())
    assert torch.equal(bits(u), bits(v)) and torch.equal(bits(s), bits(t))


def test_captured_calls_replay_on_new_inputs_and_other_streams():
    c, d = (Case([50, 14], 64, BF, s, act="gelu") for s in (19, 20))
    want = {}
    for k in (c, d):
        st = k.h0.clone()
        want[k] = (gdn.gdn_linear_recurrence_fwd(cu_seqlens=k.cu, state=st, **k.args()), st,
                   gdn.gdn_linear_recurrence_bwd(cu_seqlens=k.cu, d_out=k.dy, init_state=k.h0, **k.args()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, pool, static = torch.cuda.CUDAGraph(), c.h0.clone(), Case([50, 14], 64, BF, 19, act="gelu")
    with torch.cuda.graph(graph, stream=side):
        y = gdn.gdn_linear_recurrence_fwd(cu_seqlens=static.cu, state=pool, **static.args())
        g = gdn.gdn_linear_recurrence_bwd(cu_seqlens=static.cu, d_out=static.dy, init_state=static.h0, **static.args())
    e = Case([20, 44], 64, BF, 21, act="gelu")  # the same graph takes other lengths
    st = e.h0.clone()
    want[e] = (gdn.gdn_linear_recurrence_fwd(cu_seqlens=e.cu, state=st, **e.args()), st,
               gdn.gdn_linear_recurrence_bwd(cu_seqlens=e.cu, d_out=e.dy, init_state=e.h0, **e.args()))
    for k in (d, c, e, d):
        for n in ("x", "ag", "xg", "z", "ap", "dy", "h0", "cu"):
            getattr(static, n).copy_(getattr(k, n))
        pool.copy_(k.h0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want[k][0])) and torch.equal(bits(pool), bits(want[k][1]))
        for n in g:
            assert torch.equal(bits(g[n]), bits(want[k][2][n])), n
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2 = gdn.gdn_linear_recurrence_fwd(cu_seqlens=c.cu, state=c.h0.clone(), stream=other, **c.args())
    g2 = gdn.gdn_linear_recurrence_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, stream=other, **c.args())
    other.synchronize()
    assert torch.equal(bits(y2), bits(want[c][0]))
    for n in g2:
        assert torch.equal(bits(g2[n]), bits(want[c][2][n])), n


def test_refused_tensors():
    """What the binding refuses before it launches anything (the good call runs last)."""
    x, wide = torch.zeros(4, 16, device=DEV), torch.zeros(4, 32, device=DEV)
    cu, st = torch.tensor([0, 4], dtype=torch.int32, device=DEV), torch.zeros(2, 16, device=DEV)
    good = dict(x=x, a_gate=x, cu_seqlens=cu, state=st)
    for error, change in ((ValueError, dict(x=x[:, :8])), (ValueError, dict(a_gate=x.cpu())), (TypeError, dict(x_gate=x.bfloat16())), (ValueError, dict(z=wide[:, ::2])),
                          (ValueError, dict(x=x[:1].expand(4, 16))), (TypeError, dict(cu_seqlens=cu.long())), (ValueError, dict(a_param=x)), (ValueError, dict(state=st[:, :8])),
                          (ValueError, dict(state_indices=cu)), (TypeError, dict(x=x.half(), a_gate=x.half())), (gdn.GdnError, dict(z=torch.zeros(4, 17, device=DEV)[:, :16])),
                          (gdn.GdnError, dict(out=x)), (ValueError, dict(out=wide[:, :16])), (ValueError, dict(input_scale="square")), (ValueError, dict(activation="relu")),
                          (gdn.GdnError, dict(decay=0.0, a_param=wide[0, :16])), (ValueError, dict(cu_seqlens=cu[:0])), (TypeError, dict(a_gate=None))):
        with pytest.raises(error):
            gdn.gdn_linear_recurrence_fwd(**dict(good, **change))
    assert gdn.gdn_linear_recurrence_fwd(**good).shape == (4, 16)
