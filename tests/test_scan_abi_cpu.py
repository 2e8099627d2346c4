"""CPU checks of what the scan, the conv's gradient and the q/k norm refuse: the C entry points
return before any CUDA call, the binding raises before it reaches them."""
import ctypes

import pytest
import torch

import invariant_linear_attention_gb300 as gdn
from invariant_linear_attention_gb300 import binding

FAKE = 0x10000  # never dereferenced: every case fails validation first
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from invariant_linear_attention_gb300 import build_lib
    build_lib.build()
    return gdn.lib()


def ptrs(*names):
    return {n: FAKE + i * 0x1000 for i, n in enumerate(names)}


def scan_shape(**kw):
    base = dict(N=2, T_total=10, C=64, G=2, S=16, dtype=binding.GDN_BF16, dt_softplus=1, ldx=64, lddt=64, ldz=64, ldB=32, ldC=32)
    return gdn.ScanShape(**dict(base, **kw))


SHAPES = [(dict(S=12), UNSUPPORTED), (dict(S=128), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(G=3), INVALID), (dict(G=0), INVALID),
          (dict(C=40, G=2), UNSUPPORTED), (dict(N=-1), INVALID), (dict(ldx=60), INVALID), (dict(lddt=68), INVALID), (dict(ldB=16), INVALID),
          (dict(ldC=36), INVALID), (dict(ldz=8), INVALID), (dict(T_total=2 ** 31 - 1), UNSUPPORTED), (dict(N=1 << 26), UNSUPPORTED)]


@pytest.mark.parametrize("shape,expect", SHAPES)
def test_scan_shapes(lib, shape, expect):
    s = scan_shape(**shape)
    p = ptrs("x", "dt", "A", "B", "C", "D", "z", "b", "cu", "st", "idx", "has", "y")
    v = list(p.values())
    assert lib.gdn_selective_scan_fwd(ctypes.byref(s), *v[:11], 1 << 30, v[11], v[12], None) == expect
    u = scan_shape(**dict(dict(N=10), **shape))
    if "N" not in shape and "T_total" not in shape:
        assert lib.gdn_selective_scan_update(ctypes.byref(u), *v[:8], v[9], v[10], 64, v[12], None) == expect
    if "ldz" not in shape:
        assert lib.gdn_selective_scan_bwd_workspace_size(ctypes.byref(s)) == 0
    assert lib.gdn_selective_scan_bwd(ctypes.byref(s), *range(FAKE, FAKE + 22 * 16, 16), 1 << 40, None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(x=0), INVALID), (dict(A=0), INVALID), (dict(cu=0), INVALID), (dict(y=0), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(st=FAKE + 4), INVALID), (dict(D=FAKE + 2), INVALID), (dict(idx=FAKE + 1), INVALID), (dict(y="x"), INVALID), (dict(y="z"), INVALID),
    (dict(slots=-1), INVALID), (dict(idx=0, slots=1), INVALID)])
def test_scan_pointers(lib, change, expect):
    p = ptrs("x", "dt", "A", "B", "C", "D", "z", "b", "cu", "st", "idx", "has", "y")
    slots = change.pop("slots", 4) if "slots" in change else 4
    for k, v in change.items():
        p[k] = p[v] if isinstance(v, str) else v
    a = {k: v or None for k, v in p.items()}
    s = scan_shape()
    assert lib.gdn_selective_scan_fwd(ctypes.byref(s), a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["b"], a["cu"], a["st"],
                                      a["idx"], slots, a["has"], a["y"], None) == expect
    if "cu" not in change:
        u = scan_shape(N=10)
        slots = 9 if "idx" in change and not change["idx"] else slots
        assert lib.gdn_selective_scan_update(ctypes.byref(u), a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["b"], a["st"],
                                             a["idx"], slots, a["y"], None) == expect


def test_scan_update_needs_one_token_per_sequence_and_a_pool(lib):
    v = list(ptrs(*"abcdefghijk").values())
    assert lib.gdn_selective_scan_update(ctypes.byref(scan_shape(N=9)), *v[:8], v[8], v[9], 64, v[10], None) == INVALID
    assert lib.gdn_selective_scan_update(ctypes.byref(scan_shape(N=10)), *v[:8], None, v[9], 64, v[10], None) == INVALID
    assert lib.gdn_selective_scan_update(ctypes.byref(scan_shape(N=0, T_total=0)), *([None] * 10), 0, None, None) == 0
    assert lib.gdn_selective_scan_fwd(ctypes.byref(scan_shape(N=0)), *v, 64, None, None, None) == INVALID


BWD = ("x", "dt", "A", "B", "C", "D", "z", "b", "cu", "h0", "dy", "gT", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "ws")


@pytest.mark.parametrize("change,expect", [
    (dict(dy=0), INVALID), (dict(dx=0), INVALID), (dict(dz=0), INVALID), (dict(dA=0), INVALID), (dict(cu=0), INVALID),
    (dict(dB=FAKE + 8), INVALID), (dict(dD=FAKE + 2), INVALID), (dict(dx="x"), INVALID), (dict(ddt="dy"), INVALID), (dict(dC="B"), INVALID),
    (dict(dh0="h0"), INVALID), (dict(dh0="gT"), INVALID), (dict(ws=0), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE),
    (dict(ws_bytes=64), WORKSPACE)])
def test_scan_backward_pointers(lib, change, expect):
    p = ptrs(*BWD)
    ws = change.get("ws_bytes", 1 << 40)
    for k, v in change.items():
        if k != "ws_bytes":
            p[k] = p[v] if isinstance(v, str) else v
    s = scan_shape()
    assert lib.gdn_selective_scan_bwd(ctypes.byref(s), *(v or None for v in p.values()), ws, None) == expect
    assert lib.gdn_selective_scan_bwd_workspace_size(ctypes.byref(s)) > 0


CONV = ("x", "w", "b", "cu", "h0", "dy", "dT", "dx", "dw", "db", "dh0", "ws")


@pytest.mark.parametrize("shape,change,expect", [
    (dict(W=9), {}, UNSUPPORTED), (dict(W=1), {}, UNSUPPORTED), (dict(C=60), {}, UNSUPPORTED), (dict(dtype=3), {}, UNSUPPORTED),
    (dict(N=0), {}, INVALID), (dict(T_total=2 ** 31 - 2), {}, UNSUPPORTED), ({}, dict(x=0), INVALID), ({}, dict(w=0), INVALID),
    ({}, dict(dw=0), INVALID), ({}, dict(dx="x"), INVALID), ({}, dict(dx="dy"), INVALID), ({}, dict(dh0="dT"), INVALID),
    ({}, dict(dy=FAKE + 8), INVALID), ({}, dict(b=FAKE + 2), INVALID), ({}, dict(ws=0), WORKSPACE), ({}, dict(ws_bytes=8), WORKSPACE)])
def test_conv_backward(lib, shape, change, expect):
    p = ptrs(*CONV)
    ws = change.get("ws_bytes", 1 << 40)
    for k, v in change.items():
        if k != "ws_bytes":
            p[k] = p[v] if isinstance(v, str) else v
    s = binding.ConvShape(**dict(dict(N=2, T_total=10, C=64, W=4, dtype=binding.GDN_BF16, activation=1), **shape))
    assert lib.gdn_causal_conv1d_bwd(ctypes.byref(s), *(v or None for v in p.values()), ws, None) == expect


def qk_shape(**kw):
    base = dict(T=10, HQ=4, HK=2, d=64, rotary_dim=32, interleaved=0, norm=0, max_positions=100, eps=1e-6, dtype=binding.GDN_BF16,
                ldq=256, ldk=128)
    return gdn.QkShape(**dict(base, **kw))


QK = [(dict(d=60), UNSUPPORTED), (dict(d=512, ldq=2048, ldk=1024), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED),
      (dict(rotary_dim=80), INVALID), (dict(norm=2), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(eps=-1.0), INVALID),
      (dict(ldq=248), INVALID), (dict(ldk=132), INVALID), (dict(HQ=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("shape,expect", QK)
def test_qk_shapes(lib, shape, expect):
    s, v = qk_shape(**shape), list(ptrs(*"abcdefghijklmn").values())
    assert lib.gdn_qk_norm_rope(ctypes.byref(s), *v[:9], None) == expect
    assert lib.gdn_qk_norm_rope_bwd(ctypes.byref(s), *v[:11], 1 << 20, 1 << 20, *v[11:14], 1 << 40, None) == expect
    assert lib.gdn_qk_norm_rope_bwd_workspace_size(ctypes.byref(s)) == 0


def test_qk_pointers(lib):
    names = ("q", "k", "qw", "kw", "cos", "sin", "pos", "qo", "ko")
    for change, shape in ((dict(q=None), {}), (dict(ko=None), {}), (dict(cos=None), {}), (dict(q=FAKE + 8), {}), (dict(qw=FAKE + 4), {}),
                          (dict(pos=FAKE + 1), {}), (dict(pos=None), dict(max_positions=9)), (dict(qo="k"), {}), (dict(qo="ko"), {}),
                          (dict(qo="q"), dict(ldq=512))):
        p = ptrs(*names)
        for k, v in change.items():
            p[k] = p[v] if isinstance(v, str) else v
        assert lib.gdn_qk_norm_rope(ctypes.byref(qk_shape(**shape)), *p.values(), None) == INVALID, change
    p = ptrs("q", "k", "qw", "kw", "cos", "sin", "pos", "dqo", "dko", "dq", "dk")
    w = ptrs("dqw", "dkw", "ws")
    bwd = lambda p, w=w, ldq=256, ldk=128, ws=1 << 40: lib.gdn_qk_norm_rope_bwd(  # noqa: E731
        ctypes.byref(qk_shape()), *p.values(), ldq, ldk, *w.values(), ws, None)
    assert bwd(dict(p, dqo=None)) == INVALID and bwd(dict(p, dq=p["q"])) == INVALID and bwd(dict(p, dk=p["dq"])) == INVALID
    assert bwd(dict(p, qw=None)) == INVALID and bwd(p, ldq=248) == INVALID and bwd(p, ldk=130) == INVALID
    assert bwd(dict(p, dq=p["dqo"]), ldq=512) == INVALID
    assert bwd(p, dict(w, ws=None)) == WORKSPACE and bwd(p, ws=8) == WORKSPACE


def test_binding_refuses_before_the_library():
    x, bc, A = torch.zeros(4, 16), torch.zeros(4, 1, 8), torch.zeros(16, 8)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_selective_scan_fwd(x, x, A, bc, bc, cu)  # not on a GPU
    with pytest.raises(ValueError):
        gdn.gdn_selective_scan_fwd(x[0], x, A, bc, bc, cu)
    with pytest.raises(TypeError):
        gdn.gdn_selective_scan_update(None, x, A, bc, bc, A)
    with pytest.raises(ValueError):
        gdn.gdn_selective_scan_bwd(x, x, A, bc, bc, cu, x)
    with pytest.raises(ValueError):
        gdn.gdn_causal_conv1d_bwd(x, torch.zeros(16, 4), cu, x)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(bc, bc, A, A, norm="layer")
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope_bwd(bc, bc, A, A, bc, bc)
