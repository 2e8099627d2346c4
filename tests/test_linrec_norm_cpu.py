"""CPU checks of the gated linear recurrence and the RMSNorm with the residual's addition: the oracles
against hand-worked values and finite differences, and what the C entry points and the binding refuse
before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from invariant_linear_attention_gb300 import binding
from oracle import layer_ops
from oracle import linrec_ops as ref

FAKE = 0x10000  # never dereferenced: every case fails validation first
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from invariant_linear_attention_gb300 import build_lib
    build_lib.build()
    return gdn.lib()


# ---------------------------------------------------------------- the oracles

def test_oracle_by_hand():
    # without a_param and with gates of 0: a = 1/2; scale linear: h = (h + x) / 2; silu(0) = 0
    x = np.array([[2.0], [4.0], [8.0]])
    y, last = ref.linear_recurrence(x, np.zeros((3, 1)), [0, 2, 3], input_scale="linear")
    assert np.allclose(y[:, 0], [1.0, 2.5, 4.0]) and np.allclose(last[:, 0], [2.5, 4.0])
    y, _ = ref.linear_recurrence(x, np.zeros((3, 1)), [0, 3], input_scale="linear", z=np.zeros((3, 1)))
    assert np.all(y == 0)
    # a_param with softplus = log 2 / 4, decay 8 and an open gate of 1/2: a = e^-(log 2) = 1/2; scale sqrt: sqrt(3) / 2
    ap = np.log(np.expm1(np.log(2) / 4)).reshape(1)
    _, last = ref.linear_recurrence(x[:1], np.zeros((1, 1)), [0, 1], a_param=ap, init_state=np.array([[6.0]]))
    assert np.allclose(last, 3 + np.sqrt(3))
    # gates far out: the state is kept
    _, last = ref.linear_recurrence(x, np.full((3, 1), -800.0), [0, 3], a_param=ap, init_state=np.array([[6.0]]))
    assert np.all(last == 6)


@pytest.mark.parametrize("param", [True, False])
@pytest.mark.parametrize("scale", ["sqrt", "linear", "one"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_oracle_gradient_by_differences(param, scale, act):
    rng = np.random.default_rng(5)
    T, C, cu = 7, 3, [0, 4, 4, 6]
    a = dict(x=rng.normal(size=(T, C)), a_gate=rng.normal(size=(T, C)), init_state=rng.normal(size=(3, C)))
    if param:
        a["a_param"] = rng.normal(size=C)
    if act:
        a["z"], a["x_gate"] = rng.normal(size=(T, C)), rng.normal(size=(T, C))
    kw = dict(input_scale=scale, decay=2.0, activation=act or "silu")
    dy, gT = rng.normal(size=(T, C)), rng.normal(size=(3, C))

    def loss(v):
        y, last = ref.linear_recurrence(cu=cu, **v, **kw)
        return (y[:cu[-1]] * dy[:cu[-1]]).sum() + (last * gT).sum()

    got = ref.linear_recurrence_bwd(cu=cu, d_out=dy, d_final_state=gT, **a, **kw)
    names = dict(x="dx", a_gate="da_gate", x_gate="dx_gate", z="dz", a_param="da_param", init_state="d_init_state")
    for k, v in a.items():
        for at in np.ndindex(v.shape):
            if k not in ("a_param", "init_state") and at[0] >= cu[-1]:
                continue
            e = np.zeros(v.shape)
            e[at] = 1e-5
            assert abs((loss(dict(a, **{k: v + e})) - loss(dict(a, **{k: v - e}))) / 2e-5 - got[names[k]][at]) < 1e-7, (k, at)


def test_norm_oracle_gradient_by_differences():
    rng = np.random.default_rng(6)
    s, w, dy, dr = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    loss = lambda s, w: (layer_ops.add_rmsnorm(s, w, 0.1) * dy).sum() + (s * dr).sum()  # noqa: E731
    dx, dw = layer_ops.add_rmsnorm_bwd(s, w, dy, dr, 0.1)
    for at in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[at] = 1e-5
        assert abs((loss(s + e, w) - loss(s - e, w)) / 2e-5 - dx[at]) < 1e-8
    for i in range(5):
        e = np.zeros(5)
        e[i] = 1e-5
        assert abs((loss(s, w + e) - loss(s, w - e)) / 2e-5 - dw[i]) < 1e-8


def test_series_of_the_decay():
    """1 - e^-w below 1/4: the kernels' polynomial in float64 is within 2^-26 of the function."""
    w = np.linspace(1e-6, 0.25, 100001)
    q = 0.00767176877707243
    for c in (-0.041564859449863434, 0.1666616052389145, -0.4999999701976776):
        q = q * w + c
    assert np.abs((w + w * w * q) / -np.expm1(-w) - 1).max() < 2.0 ** -26


# ---------------------------------------------------------------- what the entry points refuse

def ptrs(*names):
    return {n: FAKE + i * 0x1000 for i, n in enumerate(names)}


def rec_shape(**kw):
    base = dict(N=2, T_total=10, C=64, dtype=binding.GDN_BF16, scale=0, activation=1, decay=8.0, ldx=64, lda=64, ldg=64, ldz=64)
    return gdn.LinrecShape(**dict(base, **kw))


FWD = ("x", "ag", "ap", "xg", "z", "cu", "st", "idx", "has", "y")
BWD = ("x", "ag", "ap", "xg", "z", "cu", "h0", "dy", "gT", "dx", "da", "dap", "dg", "dz", "dh0", "ws")


def fwd(lib, s, a, slots=4):
    return lib.gdn_linear_recurrence_fwd(ctypes.byref(s), a["x"], a["ag"], a["ap"], a["xg"], a["z"], a["cu"], a["st"], a["idx"], slots, a["has"], a["y"], None)


def update(lib, s, a, slots=64):
    return lib.gdn_linear_recurrence_update(ctypes.byref(s), a["x"], a["ag"], a["ap"], a["xg"], a["z"], a["st"], a["idx"], slots, a["y"], None)


@pytest.mark.parametrize("shape,expect", [
    (dict(dtype=7), UNSUPPORTED), (dict(scale=3), UNSUPPORTED), (dict(scale=-1), UNSUPPORTED), (dict(activation=2), UNSUPPORTED), (dict(C=60), UNSUPPORTED),
    (dict(C=0), INVALID), (dict(N=-1), INVALID), (dict(T_total=-1), INVALID), (dict(ldx=56), INVALID), (dict(lda=68), INVALID), (dict(ldg=8), INVALID),
    (dict(ldz=60), INVALID), (dict(decay=0.0), INVALID), (dict(decay=-1.0), INVALID), (dict(decay=float("inf")), INVALID),
    (dict(decay=float("nan")), INVALID), (dict(T_total=2 ** 31 - 300), UNSUPPORTED), (dict(N=1 << 26), UNSUPPORTED)])
def test_recurrence_shapes(lib, shape, expect):
    s, a = rec_shape(**shape), ptrs(*FWD)
    assert fwd(lib, s, a) == expect
    if "N" not in shape and "T_total" not in shape:
        assert update(lib, rec_shape(**dict(dict(N=10), **shape)), a) == expect
    assert lib.gdn_linear_recurrence_bwd(ctypes.byref(s), *ptrs(*BWD).values(), 1 << 40, None) == expect
    if not set(shape) & {"ldg", "ldz", "decay", "activation"}:
        assert lib.gdn_linear_recurrence_bwd_workspace_size(ctypes.byref(s)) == 0


@pytest.mark.parametrize("C", [2 ** 31 - 8, 2 ** 31 - 32])
@pytest.mark.parametrize("N", [0, 1])
def test_recurrence_channels_at_the_end_of_31_bits(lib, C, N):
    """Blocks of 32 channels are counted in 31 bits: refused, not launched with a count that has passed them."""
    a = ptrs(*FWD)
    wide = dict(N=N, T_total=N, C=C, ldx=C, lda=C, ldg=C, ldz=C)
    assert fwd(lib, rec_shape(**wide), a) == UNSUPPORTED and update(lib, rec_shape(**wide), a) == UNSUPPORTED
    assert lib.gdn_linear_recurrence_bwd(ctypes.byref(rec_shape(**wide)), *ptrs(*BWD).values(), 1 << 62, None) == UNSUPPORTED
    assert lib.gdn_linear_recurrence_bwd_workspace_size(ctypes.byref(rec_shape(**wide))) == 0
    fits = dict(dict.fromkeys(("C", "ldx", "lda", "ldg", "ldz"), 2 ** 31 - 72), N=1, T_total=1)
    assert lib.gdn_linear_recurrence_bwd_workspace_size(ctypes.byref(rec_shape(**fits))) == 16 * (2 ** 31 - 72)


@pytest.mark.parametrize("change,expect", [
    (dict(x=0), INVALID), (dict(ag=0), INVALID), (dict(cu=0), INVALID), (dict(y=0), INVALID), (dict(x=FAKE + 8), INVALID), (dict(ap=FAKE + 4), INVALID),
    (dict(st=FAKE + 4), INVALID), (dict(idx=FAKE + 1), INVALID), (dict(y="x"), INVALID), (dict(y="ag"), INVALID), (dict(y="xg"), INVALID),
    (dict(y="z"), INVALID), (dict(slots=-1), INVALID), (dict(idx=0, slots=1), INVALID), (dict(has=FAKE + 2), INVALID)])
def test_recurrence_pointers(lib, change, expect):
    p = ptrs(*FWD)
    slots = change.get("slots", 4)
    for k, v in change.items():
        if k != "slots":
            p[k] = p[v] if isinstance(v, str) else v
    a = {k: v or None for k, v in p.items()}
    assert fwd(lib, rec_shape(), a, slots) == expect
    if "cu" not in change and "has" not in change:
        assert update(lib, rec_shape(N=10), a, 9 if "idx" in change and not change["idx"] else slots) == expect


def test_recurrence_update_needs_one_token_per_sequence_and_a_pool(lib):
    a = ptrs(*FWD)
    assert update(lib, rec_shape(N=9), a) == INVALID
    assert update(lib, rec_shape(N=10), dict(a, st=None)) == INVALID
    assert update(lib, rec_shape(N=0, T_total=0), dict.fromkeys(a)) == 0
    assert fwd(lib, rec_shape(N=0), a) == INVALID
    assert fwd(lib, rec_shape(N=0, T_total=0), dict.fromkeys(a)) == 0


@pytest.mark.parametrize("change,expect", [
    (dict(dy=0), INVALID), (dict(dx=0), INVALID), (dict(da=0), INVALID), (dict(dg=0), INVALID), (dict(dz=0), INVALID), (dict(cu=0), INVALID),
    (dict(da=FAKE + 8), INVALID), (dict(dap=FAKE + 2), INVALID), (dict(h0=FAKE + 4), INVALID), (dict(dx="x"), INVALID), (dict(da="dy"), INVALID),
    (dict(dg="z"), INVALID), (dict(dz="da"), INVALID), (dict(ap=0), INVALID), (dict(dh0="h0"), INVALID), (dict(dh0="gT"), INVALID), (dict(ws=0), WORKSPACE),
    (dict(ws=FAKE + 8), WORKSPACE), (dict(ws_bytes=8), WORKSPACE)])
def test_recurrence_backward_pointers(lib, change, expect):
    p = ptrs(*BWD)
    for k, v in change.items():
        if k != "ws_bytes":
            p[k] = p[v] if isinstance(v, str) else v
    s = rec_shape()
    assert lib.gdn_linear_recurrence_bwd(ctypes.byref(s), *(v or None for v in p.values()), change.get("ws_bytes", 1 << 40), None) == expect
    assert lib.gdn_linear_recurrence_bwd_workspace_size(ctypes.byref(s)) > 0


@pytest.mark.parametrize("T,N,C,dtype", [(100, 3, 64, binding.GDN_BF16), (0, 5, 8, binding.GDN_F32), (1 << 20, 1, 4096, binding.GDN_BF16), (2 ** 31 - 5000, 1, 8, binding.GDN_F32)])
def test_recurrence_workspace_follows_the_tokens_and_the_sequences(lib, T, N, C, dtype):
    s = rec_shape(T_total=T, N=N, C=C, dtype=dtype, ldx=C, lda=C, ldg=C, ldz=C)
    assert lib.gdn_linear_recurrence_bwd_workspace_size(ctypes.byref(s)) == 16 * (T // 32 + N) * C


def norm_shape(**kw):
    return gdn.AddNormShape(**dict(dict(rows=10, d=64, dtype=binding.GDN_BF16, eps=1e-6, group=32, ldx=64, ldr=64), **kw))


def norm_calls(lib, s, p, scales=FAKE + 0x9000):
    v = [p[k] for k in ("x", "res", "w", "ro", "y")]
    return lib.gdn_add_rmsnorm(ctypes.byref(s), *v, None), lib.gdn_add_rmsnorm_fp8(ctypes.byref(s), *v, scales, None)


@pytest.mark.parametrize("shape,expect", [
    (dict(d=60), UNSUPPORTED), (dict(d=16392, ldx=16392, ldr=16392), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(d=0), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(ldx=56), INVALID), (dict(ldx=68), INVALID)])
def test_norm_shapes(lib, shape, expect):
    s = norm_shape(**shape)
    assert norm_calls(lib, s, ptrs("x", "res", "w", "ro", "y")) == (expect, expect)
    v = list(ptrs(*"abcdefg").values())
    assert lib.gdn_add_rmsnorm_bwd(ctypes.byref(s), *v, 1 << 40, None) == expect
    assert lib.gdn_add_rmsnorm_bwd_workspace_size(ctypes.byref(s)) == 0


def test_norm_pointers(lib):
    p = ptrs("x", "res", "w", "ro", "y")
    for change, shape in ((dict(x=None), {}), (dict(w=None), {}), (dict(y=None), {}), (dict(ro=None), {}), (dict(x=FAKE + 8), {}), (dict(w=FAKE + 4), {}),
                          (dict(ro=FAKE + 0x3008), {}), (dict(), dict(ldr=56)), (dict(), dict(ldr=100)), (dict(ro=p["y"]), {}),
                          (dict(ro=p["x"]), dict(ldx=128)), (dict(ro=p["res"]), dict(ldr=128))):
        assert norm_calls(lib, norm_shape(**shape), dict(p, **change)) == (INVALID, INVALID), (change, shape)
    s = norm_shape()
    assert norm_calls(lib, norm_shape(ldx=128), dict(p, y=p["x"]))[0] == INVALID
    assert norm_calls(lib, norm_shape(group=16), p)[1] == UNSUPPORTED and norm_calls(lib, norm_shape(group=-32), p)[1] == UNSUPPORTED
    assert norm_calls(lib, s, p, None)[1] == INVALID and norm_calls(lib, s, p, FAKE + 2)[1] == INVALID
    for same in ("x", "res", "y", "ro"):
        assert norm_calls(lib, s, p, p[same])[1] == INVALID
    for same in ("x", "res"):
        assert norm_calls(lib, s, dict(p, y=p[same]))[1] == INVALID
    b = ptrs("s", "w", "dy", "dr", "dx", "dw", "ws")
    bwd = lambda b, ws=1 << 40, **kw: lib.gdn_add_rmsnorm_bwd(ctypes.byref(norm_shape(**kw)), *b.values(), ws, None)  # noqa: E731
    for change in (dict(s=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dx=FAKE + 8), dict(dw=FAKE + 4), dict(dr=FAKE + 2)):
        assert bwd(dict(b, **change)) == INVALID, change
    assert bwd(dict(b, dx=b["s"]), ldx=128) == INVALID
    assert bwd(dict(b, ws=None)) == WORKSPACE and bwd(b, 64) == WORKSPACE and bwd(dict(b, ws=FAKE + 8)) == WORKSPACE


def test_binding_refuses_before_the_library():
    x, w, cu = torch.zeros(4, 16), torch.zeros(16), torch.zeros(2, dtype=torch.int32)
    for error, call in ((ValueError, lambda: gdn.gdn_linear_recurrence_fwd(x, x, cu)), (TypeError, lambda: gdn.gdn_linear_recurrence_fwd(None, x, cu)),
                        (ValueError, lambda: gdn.gdn_linear_recurrence_update(x, x, x)), (ValueError, lambda: gdn.gdn_linear_recurrence_bwd(x, x, cu, x)),
                        (ValueError, lambda: gdn.gdn_add_rmsnorm(x, w)), (TypeError, lambda: gdn.gdn_add_rmsnorm(None, w)),
                        (ValueError, lambda: gdn.gdn_add_rmsnorm_fp8(x, w)), (ValueError, lambda: gdn.gdn_add_rmsnorm_bwd(x, w, x))):
        with pytest.raises(error):
            call()


def test_norm_gradient_of_no_rows_needs_the_weight_of_dweight(lib):
    """With no rows dweight is still written, by a kernel that reads the weight; without dweight there is nothing to do."""
    b = ptrs("s", "w", "dy", "dr", "dx", "dw", "ws")
    for d, dtype in ((64, binding.GDN_BF16), (4, binding.GDN_F32), (16384, binding.GDN_BF16)):
        s = norm_shape(rows=0, d=d, dtype=dtype, ldx=d)
        assert lib.gdn_add_rmsnorm_bwd(ctypes.byref(s), *dict(b, w=None).values(), 1 << 40, None) == INVALID
        assert lib.gdn_add_rmsnorm_bwd(ctypes.byref(s), *dict.fromkeys(b, None).values(), 0, None) == 0


def test_norm_output_alignment(lib):
    """8 bytes for y in 8 bits, 16 in the input's type."""
    p = ptrs("x", "res", "w", "ro", "y")
    for off in (1, 2, 4, 12):
        assert norm_calls(lib, norm_shape(), dict(p, y=p["y"] + off)) == (INVALID, INVALID)
    v = [dict(p, y=p["y"] + 8)[k] for k in ("x", "res", "w", "ro", "y")]
    assert lib.gdn_add_rmsnorm(ctypes.byref(norm_shape()), *v, None) == INVALID
