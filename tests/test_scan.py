"""GPU parity, invariance and gradients of the selective scan against the fp64 oracle
(oracle/scan_ops.py).

Tolerances, in units of u = 2^-24 of the sum of the terms' magnitudes M (the oracle run on
absolute values).  The step d = softplus(v), |v| < 13 here, carries its exponential's argument
rounding (2 |v| u), the hardware exponential (2^-22) and about a dozen roundings: below 46 u.
A decay's exponential carries 4 u plus its argument's relative error (46 u for d, 6 u for A)
times the argument; over the k <= L tokens between a term and its use that adds to at most
4 L u + 52 u s, where s = sum of d |A| in between (past s = 40 the term is below e^-40 of
itself).  With the products and sums of a token (2 u each, L of them) and those over the states
(S / 4 + 6) and the skip term:
    E = 64 + 6 L + 52 min(40, max over channels of sum d |A|) + S / 4.
The gate adds (6 + 2.4 |z|) u of the result.  A gradient multiplies two such recurrences (2 E)
and three more products; sums over channels or tokens add one rounding each (C or T): 3 E + C + T.
The gate's slope p (1 + z (1 - p)), p = sigmoid(z), is a sum that cancels near z = -1.28: with p's
relative error E_p = (7 + 2.4 |z|) u its absolute error is at most
p (E_p |1 + z (1 - p)| + |z| p E_p + 2 u (1 + |z|)) <= (E_p + 2 u) p (1 + |z|): the oracle's
magnitude of dz takes p (1 + |z|) for the slope, and E_p + 2 u is within the 3 (6 + 2.4 |z|) u that
the gate adds to a gradient.
A bf16 output adds its own rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from oracle import scan_ops as ref
from helpers import BF16_ROUND, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
LENS = [33, 0, 1, 70, 16, 2, 8, 31]


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def rounding(dtype):
    return BF16_ROUND if dtype == torch.bfloat16 else U


class Case:
    """Inputs of a ragged batch; x, z, B and C as columns of wider rows when strided."""

    def __init__(self, lens, C, G, S, dtype, seed, gate=True, D=True, bias=True, strided=False, behind=0, slow=False):
        gen = torch.Generator().manual_seed(seed)
        T = sum(lens) + behind
        rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731

        def rows(n, *shape):
            wide = rn(n, int(np.prod(shape)) + (24 if strided else 0)).to(dtype).to(DEV)
            return (wide[:, 8:-16] if strided else wide).unflatten(1, shape) if len(shape) > 1 else (wide[:, 8:-16] if strided else wide)

        self.lens, self.C, self.G, self.S, self.dtype = lens, C, G, S, dtype
        self.cu_list = np.concatenate([[0], np.cumsum(lens)]).tolist()
        self.cu = torch.tensor(self.cu_list, dtype=torch.int32, device=DEV)
        self.x, self.dt = rows(T, C), rows(T, C)
        self.z = rows(T, C) if gate else None
        self.B, self.Cm = rows(T, G, S), rows(T, G, S)
        self.A_log = (torch.log(torch.rand(C, S, generator=gen) * (0.05 if slow else 8) + 1e-3)).to(DEV)
        self.D = rn(C).to(DEV) if D else None
        self.bias = (rn(C) - 3).to(DEV) if bias else None
        self.dy = rn(T, C).to(dtype).to(DEV)
        self.h0, self.gT = rn(len(lens), C, S).to(DEV), rn(len(lens), C, S).to(DEV)

    def args(self, t=slice(None)):
        return dict(x=self.x[t], dt=self.dt[t], A_log=self.A_log, B=self.B[t], C=self.Cm[t], D=self.D,
                    z=None if self.z is None else self.z[t], dt_bias=self.bias)

    def error_units(self):
        raw = to_np(self.dt) + (0 if self.bias is None else to_np(self.bias))
        assert np.abs(raw).max() < 13
        d, A = ref.softplus(raw), np.exp(to_np(self.A_log))
        s = max((d[a:b].sum(0)[:, None] * A).max() for a, b in zip(self.cu_list, self.cu_list[1:]))
        return 64 + 6 * max(self.lens) + 52 * min(40.0, s) + self.S / 4


GRID = [(torch.bfloat16, 16, 1, 200, True), (torch.float32, 16, 1, 72, True), (torch.float32, 8, 2, 272, False),
        (torch.bfloat16, 32, 3, 120, False), (torch.float32, 64, 1, 40, True), (torch.bfloat16, 64, 2, 16, False),
        (torch.bfloat16, 8, 1, 8, True)]


def check(got, want, mag, units, dtype, extra=0.0):
    got = to_np(got)
    assert np.all(np.isnan(got) == np.isnan(want)) if np.isnan(want).any() else True
    ok = ~np.isnan(want)
    bound = units * U * (mag if np.ndim(mag) == 0 else mag[ok]) + (rounding(dtype) + extra * U) * np.abs(want[ok]) + 1e-30
    err = np.abs(got[ok] - want[ok])
    assert np.all(err <= bound), (err / bound).max()


@pytest.mark.parametrize("dtype,S,G,C,gate", GRID)
@pytest.mark.parametrize("strided", [False, True])
def test_forward_vs_oracle(dtype, S, G, C, gate, strided):
    c = Case(LENS, C, G, S, dtype, 11, gate=gate, D=gate, bias=gate or strided, strided=strided, behind=3, slow=strided)
    N = len(LENS)
    pool0 = torch.randn(N + 4, C, S, generator=torch.Generator().manual_seed(1)).to(DEV)
    slots = torch.randperm(N + 4, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
    has = torch.tensor([1, 1, 0, 1, 0, 1, 1, 0], dtype=torch.int32)
    pool = pool0.clone()
    out = torch.full((sum(LENS) + 3, C), float("nan"), dtype=dtype, device=DEV)
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, state_indices=slots.to(DEV), has_initial_state=has.to(DEV), out=out,
                                   **c.args())
    assert y is out
    init = to_np(pool0)[slots.long().numpy()] * has.numpy()[:, None, None]
    want, fin = ref.selective_scan(cu=c.cu_list, init_state=init, **c.args())
    absargs = {k: None if v is None else v.abs() if k in ("x", "B", "C", "D") else v for k, v in c.args().items()}
    mag, fmag = ref.selective_scan(cu=c.cu_list, init_state=np.abs(init), **dict(absargs, z=None))
    gate_units = 0.0
    if gate:
        mag = mag * np.abs(ref.silu(to_np(c.z)))
        gate_units = 6 + 2.4 * np.abs(to_np(c.z)).max()
    check(y, want, mag, c.error_units(), dtype, gate_units)
    got = to_np(pool)
    assert np.all(np.abs(got[slots.long().numpy()] - fin) <= (c.error_units() + 1) * U * fmag + 1e-30)
    spare = sorted(set(range(N + 4)) - set(slots.tolist()))
    assert torch.equal(bits(pool[spare]), bits(pool0[spare]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,C", [(16, 136), (8, 16), (64, 24), (32, 520)])
def test_bits_do_not_depend_on_the_batch_or_on_how_tokens_arrive(dtype, S, C):
    lens = [77, 5, 130, 1]
    c = Case(lens, C, 1, S, dtype, 12)
    pool = c.h0.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    one = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    # alone
    for n in (0, 2):
        t = slice(c.cu_list[n], c.cu_list[n + 1])
        st = c.h0[n:n + 1].clone()
        alone = gdn.gdn_selective_scan_fwd(cu_seqlens=one(lens[n]), state=st, **c.args(t))
        assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(st[0]), bits(pool[n]))
    # in three chained calls, the last tokens one by one beside another sequence
    a = c.cu_list[2]
    st = torch.zeros(3, C, S, device=DEV)
    st[2] = c.h0[2]
    idx = torch.tensor([2], dtype=torch.int32, device=DEV)
    parts = [gdn.gdn_selective_scan_fwd(cu_seqlens=one(m - k), state=st, state_indices=idx, **c.args(slice(a + k, a + m)))
             for k, m in ((0, 33), (33, 34), (34, 120))]
    both = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    for t in range(120, 130):
        rows = torch.tensor([a + t, t], device=DEV)
        parts.append(gdn.gdn_selective_scan_update(state=st, state_indices=both, **c.args(rows))[:1])
    assert torch.equal(bits(torch.cat(parts)), bits(y[a:a + 130]))
    assert torch.equal(bits(st[2]), bits(pool[2]))


@pytest.mark.parametrize("dtype,S,G,C,gate", [(torch.bfloat16, 16, 1, 2056, True), (torch.float32, 16, 2, 592, False), (torch.bfloat16, 8, 3, 1056, False),
                                              (torch.float32, 8, 1, 1032, True), (torch.bfloat16, 32, 1, 264, True),
                                              (torch.float32, 32, 2, 272, False), (torch.bfloat16, 64, 1, 136, False), (torch.float32, 64, 2, 144, True),
                                              (torch.float32, 16, 2, 1040, False), (torch.bfloat16, 32, 1, 520, True), (torch.float32, 32, 2, 528, False),
                                              (torch.bfloat16, 64, 1, 264, False), (torch.float32, 64, 2, 272, True)])
def test_large_batches_agree_with_a_sequence_alone(dtype, S, G, C, gate):
    # several CTAs an SM, sequences in order of length; then also two channels a lane
    lens = [(37 * i) % 130 for i in range(110)]
    c = Case(lens, C, G, S, dtype, 13, gate=gate, D=gate, bias=not gate)
    pool = c.h0.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, **c.args())
    for n in range(110):
        t = slice(c.cu_list[n], c.cu_list[n + 1])
        st = c.h0[n:n + 1].clone()
        cu = torch.tensor([0, lens[n]], dtype=torch.int32, device=DEV)
        alone = gdn.gdn_selective_scan_fwd(cu_seqlens=cu, state=st, **c.args(t))
        assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(st[0]), bits(pool[n])), n


@pytest.mark.parametrize("N", [100, 255, 256, 257, 300])
def test_many_sequences_of_equal_and_no_length(N):
    # equal lengths, empty sequences, slots in reverse; up to 256 sequences of these lengths are taken in order of length
    lens = [(90, 280, 280, 420)[i % 4] if i % 64 != 5 else 0 for i in range(N)]
    c = Case(lens, 72, 1, 16, torch.bfloat16, 17)
    pool = c.h0.clone()
    idx = torch.arange(N - 1, -1, -1, dtype=torch.int32, device=DEV)
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, state_indices=idx, **c.args())
    for n in (0, 1, 2, 3, 4, N // 2, N - 3, N - 2, N - 1):
        t = slice(c.cu_list[n], c.cu_list[n + 1])
        st = c.h0[N - 1 - n:N - n].clone()
        cu = torch.tensor([0, lens[n]], dtype=torch.int32, device=DEV)
        alone = gdn.gdn_selective_scan_fwd(cu_seqlens=cu, state=st, **c.args(t))
        assert torch.equal(bits(alone), bits(y[t])) and torch.equal(bits(st[0]), bits(pool[N - 1 - n])), n


@pytest.mark.parametrize("dtype,S,B,C", [(torch.bfloat16, 16, 300, 4160), (torch.float32, 8, 150, 4160), (torch.float32, 64, 37, 1000)])
def test_large_updates_agree_with_prompts_of_one_token(dtype, S, B, C):
    c = Case([1] * B, C, 1, S, dtype, 24)
    a, b = c.h0.clone(), c.h0.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=a, **c.args())
    z = gdn.gdn_selective_scan_update(state=b, **c.args())
    assert torch.equal(bits(y), bits(z)) and torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("dtype,S,G,C,gate", GRID)
def test_update_vs_oracle_and_skips(dtype, S, G, C, gate):
    B = 11
    c = Case([1] * B, C, G, S, dtype, 14, gate=gate, D=gate, bias=gate, strided=True)
    idx = torch.tensor([3, -1, 0, 12, 7, 13, 5, 1, 2, 9, 4], dtype=torch.int32, device=DEV)  # -1 and 13: skipped
    pool0 = torch.randn(13, C, S, device=DEV)
    pool, out = pool0.clone(), torch.full((B, C), 7.0, dtype=dtype, device=DEV)
    gdn.gdn_selective_scan_update(state=pool, state_indices=idx, out=out, **c.args())
    keep = [i for i in range(B) if 0 <= int(idx[i]) < 13]
    slot = idx[keep].long()
    want, fin = ref.selective_scan(cu=list(range(len(keep) + 1)), init_state=pool0[slot], **c.args(torch.tensor(keep, device=DEV)))
    absargs = {k: None if v is None else v.abs() if k in ("x", "B", "C", "D") else v for k, v in c.args(torch.tensor(keep, device=DEV)).items()}
    mag, fmag = ref.selective_scan(cu=list(range(len(keep) + 1)), init_state=pool0[slot].abs(), **dict(absargs, z=None))
    extra = 0.0
    if gate:
        zk = to_np(c.z)[keep]
        mag, extra = mag * np.abs(ref.silu(zk)), 6 + 2.4 * np.abs(zk).max()
    check(out[keep], want, mag, c.error_units(), dtype, extra)
    assert np.all(np.abs(to_np(pool[slot]) - fin) <= (c.error_units() + 1) * U * fmag + 1e-30)
    skipped = [i for i in range(B) if i not in keep]
    assert torch.all(out[skipped] == 7)
    spare = sorted(set(range(13)) - set(slot.tolist()))
    assert torch.equal(bits(pool[spare]), bits(pool0[spare]))


def test_steps_without_softplus_and_far_steps():
    c = Case([20, 9], 16, 1, 8, torch.float32, 15, bias=False)
    c.dt = torch.rand(29, 16, generator=torch.Generator().manual_seed(3)).to(DEV)
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, dt_softplus=False, **c.args())
    want, _ = ref.selective_scan(cu=c.cu_list, dt_softplus=False, **c.args())
    assert np.abs(to_np(y) - want).max() <= 1e-4 * np.abs(want).max()
    # softplus far on both sides: d = v above, e^v below (its relative error: 2 |v| u + 16 u)
    v = torch.tensor([[-60.0, -30.0, -20.0, -5.0, 0.0, 5.0, 20.0, 60.0]], device=DEV)
    one = torch.ones(1, 8, device=DEV)
    st = torch.zeros(1, 8, 8, device=DEV)
    gdn.gdn_selective_scan_update(one, v, torch.full((8, 8), -80.0, device=DEV), torch.ones(1, 1, 8, device=DEV),
                                  torch.ones(1, 1, 8, device=DEV), st)
    d = ref.softplus(to_np(v))[0]
    assert np.all(np.abs(to_np(st)[0] - d[:, None]) <= ((2 * np.abs(to_np(v)[0]) + 16) * U * d)[:, None])


def test_rows_behind_the_last_sequence_are_neither_read_nor_written():
    c = Case([40, 3], 64, 1, 16, torch.bfloat16, 16, behind=5)
    for t in (c.x, c.dt, c.z, c.B, c.Cm, c.dy):
        t[43:] = float("nan")
    out = torch.full((48, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, out=out, **c.args())
    assert torch.all(out[43:] == 3) and torch.isfinite(out[:43]).all()
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, **c.args())
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        assert torch.isfinite(g[k][:43]).all(), k
    for k in ("dA_log", "dD", "ddt_bias", "d_init_state"):
        assert torch.isfinite(g[k]).all(), k


@pytest.mark.parametrize("dtype,S,G,C,gate", GRID)
@pytest.mark.parametrize("states", [False, True])
def test_backward_vs_oracle(dtype, S, G, C, gate, states):
    c = Case(LENS, C, G, S, dtype, 17, gate=gate, D=gate or states, bias=gate or states, strided=states, slow=not states)
    st = dict(init_state=c.h0, d_final_state=c.gT) if states else {}
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, need_d_init_state=states, **st, **c.args())
    want = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, **st, **c.args())
    mag = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, magnitude=True, **st, **c.args())
    units = 3 * c.error_units() + C + sum(LENS) + (0 if not gate else 3 * (6 + 2.4 * np.abs(to_np(c.z)).max()))
    for k in ("dx", "ddt", "dB", "dC", "dA_log") + (("dz",) if gate else ()) + (("d_init_state",) if states else ()) + \
            (("dD", "ddt_bias") if c.D is not None else ()):
        wide = k in ("dA_log", "dD", "ddt_bias", "d_init_state")
        assert g[k].dtype == (torch.float32 if wide else dtype)
        check(g[k], want[k], mag[k], units, torch.float32 if wide else dtype)
    assert (g["dz"] is None) == (not gate) and (g["dD"] is None) == (c.D is None) and (g["d_init_state"] is None) == (not states)


@pytest.mark.parametrize("dtype,S,G,C,lens", [(torch.float32, 8, 64, 512, [390, 0, 150, 64, 1]), (torch.bfloat16, 16, 56, 448, [390, 0, 150, 64, 1]),
                                              (torch.float32, 8, 500, 4000, [270, 0, 130]), (torch.bfloat16, 16, 16, 128, [390, 0, 150, 64, 1]),
                                              (torch.bfloat16, 16, 320, 2560, [270, 0, 130]), (torch.float32, 64, 28, 224, [390, 0, 150, 64, 1]), (torch.bfloat16, 64, 44, 352, [390, 0, 150, 64, 1])])
def test_backward_of_a_batch_with_many_ctas(dtype, S, G, C, lens):
    # enough channel blocks and tokens for the longer segments, sequences of several of them
    c = Case(lens, C, G, S, dtype, 23, slow=True)
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    want = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    mag = ref.selective_scan_bwd(cu=c.cu_list, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, magnitude=True, **c.args())
    units = 3 * c.error_units() + C + sum(lens) + 3 * (6 + 2.4 * np.abs(to_np(c.z)).max())
    for k in want:
        kind = torch.float32 if g[k].dtype == torch.float32 else dtype
        check(g[k], want[k], mag[k], units, kind)


def test_backward_repeats_its_bits_and_takes_a_callers_workspace():
    c = Case([300, 41, 0, 7], 200, 1, 16, torch.bfloat16, 18)
    a = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, **c.args())
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    b = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, workspace=ws, **c.args())
    for k in a:
        assert torch.equal(bits(a[k]), bits(b[k])), k
    with pytest.raises(gdn.GdnError):
        gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, workspace=ws[:64], **c.args())


def test_no_tokens():
    x = torch.empty(0, 16, device=DEV)
    bc = torch.empty(0, 1, 8, device=DEV)
    A = torch.zeros(16, 8, device=DEV)
    st = torch.randn(3, 16, 8, device=DEV)
    s0, cu = st.clone(), torch.zeros(4, dtype=torch.int32, device=DEV)
    has = torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)
    y = gdn.gdn_selective_scan_fwd(x, x, A, bc, bc, cu, state=st, has_initial_state=has)
    assert y.shape == (0, 16) and torch.equal(st[[0, 2]], s0[[0, 2]]) and torch.all(st[1] == 0)
    gT = torch.randn(3, 16, 8, device=DEV)
    g = gdn.gdn_selective_scan_bwd(x, x, A, bc, bc, cu, x, d_final_state=gT)
    assert torch.equal(g["d_init_state"], gT) and torch.all(g["dA_log"] == 0)
    g = gdn.gdn_selective_scan_bwd(x, x, A, bc, bc, cu[:1], x)
    assert g["d_init_state"].shape == (0, 16, 8) and torch.all(g["dA_log"] == 0)
    assert gdn.gdn_selective_scan_update(x, x, A, bc, bc, st).shape == (0, 16)


def test_padding_only_and_slots_outside_the_pool():
    """Tokens of which no sequence has any; slots that are not in the pool."""
    c = Case([0, 0], 16, 1, 8, torch.float32, 25, behind=5)
    for t in (c.x, c.dt, c.z, c.B, c.Cm, c.dy):
        t[:] = float("nan")
    st = c.h0.clone()
    out = torch.full((5, 16), 3.0, device=DEV)
    gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=st, out=out, **c.args())
    assert torch.all(out == 3) and torch.equal(st, c.h0)
    g = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, d_final_state=c.gT, **c.args())
    assert torch.equal(g["d_init_state"], c.gT)
    for k in ("dA_log", "dD", "ddt_bias"):
        assert torch.all(g[k] == 0), k
    c = Case([9, 4, 6], 16, 1, 8, torch.float32, 26)
    pool = torch.randn(3, 16, 8, device=DEV)
    p0 = pool.clone()
    y = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=pool, state_indices=torch.tensor([-1, 3, 1 << 30], dtype=torch.int32, device=DEV),
                                   **c.args())
    assert torch.equal(y, gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, **c.args())) and torch.equal(pool, p0)


def test_captured_calls_replay_on_new_inputs_and_other_streams():
    c = Case([50, 14], 64, 1, 16, torch.bfloat16, 19)
    d = Case([30, 34], 64, 1, 16, torch.bfloat16, 20)
    pool = c.h0.clone()
    want = {}
    for k in (c, d):
        st = k.h0.clone()
        want[k] = (gdn.gdn_selective_scan_fwd(cu_seqlens=k.cu, state=st, **k.args()), st,
                   gdn.gdn_selective_scan_bwd(cu_seqlens=k.cu, d_out=k.dy, init_state=k.h0, **k.args()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    names = ("x", "dt", "z", "B", "Cm", "A_log", "D", "bias", "dy", "h0", "cu")
    static = Case([50, 14], 64, 1, 16, torch.bfloat16, 19)
    with torch.cuda.graph(graph, stream=side):
        y = gdn.gdn_selective_scan_fwd(cu_seqlens=static.cu, state=pool, **static.args())
        g = gdn.gdn_selective_scan_bwd(cu_seqlens=static.cu, d_out=static.dy, init_state=static.h0, **static.args())
    for k in (d, c, d):
        for n in names:
            getattr(static, n).copy_(getattr(k, n))
        pool.copy_(k.h0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want[k][0])) and torch.equal(bits(pool), bits(want[k][1]))
        for n in g:
            assert torch.equal(bits(g[n]), bits(want[k][2][n])), n
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2 = gdn.gdn_selective_scan_fwd(cu_seqlens=c.cu, state=c.h0.clone(), stream=other, **c.args())
    g2 = gdn.gdn_selective_scan_bwd(cu_seqlens=c.cu, d_out=c.dy, init_state=c.h0, stream=other, **c.args())
    other.synchronize()
    assert torch.equal(bits(y2), bits(want[c][0]))
    for n in g2:
        assert torch.equal(bits(g2[n]), bits(want[c][2][n])), n


def test_refused_tensors():
    """What the binding refuses before it launches anything (the good call runs last)."""
    x, bc, A = torch.zeros(4, 16, device=DEV), torch.zeros(4, 1, 8, device=DEV), torch.zeros(16, 8, device=DEV)
    cu, st = torch.tensor([0, 4], dtype=torch.int32, device=DEV), torch.zeros(2, 16, 8, device=DEV)
    good = dict(x=x, dt=x, A_log=A, B=bc, C=bc, cu_seqlens=cu, state=st)
    wide = torch.zeros(4, 32, device=DEV)
    for error, change in ((ValueError, dict(x=x[:, :8])), (ValueError, dict(dt=x.cpu())), (TypeError, dict(B=bc.bfloat16())),
                          (ValueError, dict(z=wide[:, ::2])), (ValueError, dict(x=x[:1].expand(4, 16))), (TypeError, dict(cu_seqlens=cu.long())),
                          (ValueError, dict(A_log=A.t().contiguous().t())), (ValueError, dict(state=st[:, :8])),
                          (ValueError, dict(state_indices=cu)), (TypeError, dict(x=x.half(), dt=x.half(), B=bc.half(), C=bc.half())),
                          (gdn.GdnError, dict(z=torch.zeros(4, 17, device=DEV)[:, :16])), (gdn.GdnError, dict(out=x)),
                          (ValueError, dict(out=wide[:, :16])), (ValueError, dict(D=A[:, 0])), (TypeError, dict(C=None)),
                          (ValueError, dict(cu_seqlens=cu[:0]))):
        with pytest.raises(error):
            gdn.gdn_selective_scan_fwd(**dict(good, **change))
    assert gdn.gdn_selective_scan_fwd(**good).shape == (4, 16)
