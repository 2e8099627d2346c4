"""CPU pins of the oracles of the scan, the conv's gradient and the q/k norm with rotation:
hand-worked values, and every gradient against central differences of its forward."""
import numpy as np
import pytest

from oracle import layer_ops as L
from oracle import scan_ops as S


def differences(f, arrays, names, grads, rng, points=6, step=1e-6, tol=2e-6):
    """Central differences of the scalar f(**arrays) at random points of every named array."""
    for name in names:
        a = arrays[name]
        for _ in range(points):
            at = tuple(rng.integers(0, n) for n in a.shape)
            keep = a[at]
            a[at] = keep + step
            up = f(**arrays)
            a[at] = keep - step
            down = f(**arrays)
            a[at] = keep
            want = (up - down) / (2 * step)
            got = grads[name][at]
            assert abs(got - want) <= tol * max(1.0, abs(want)), (name, at, got, want)


def test_scan_by_hand():
    # one channel, one state: d = softplus(0) = ln 2, A = -1, so a = 1/2; h: ln2, ln2/2 + 2 ln2
    ln2 = np.log(2.0)
    y, fin = S.selective_scan(np.array([[1.0], [2.0]]), np.zeros((2, 1)), np.zeros((1, 1)), np.ones((2, 1, 1)),
                              np.array([[[1.0]], [[3.0]]]), [0, 2], D=np.array([10.0]))
    assert np.allclose(y[:, 0], [ln2 + 10.0, 3 * 2.5 * ln2 + 20.0])
    assert np.allclose(fin[0], 2.5 * ln2)


@pytest.mark.parametrize("gate,softplus", [(True, True), (False, False)])
def test_scan_gradient_is_the_difference(gate, softplus):
    rng = np.random.default_rng(1)
    T, C, G, K, cu = 9, 4, 2, 3, [0, 5, 5, 9]
    a = dict(x=rng.normal(size=(T, C)), dt=rng.normal(size=(T, C)) * 0.5 + (0 if softplus else 1), A_log=rng.normal(size=(C, K)) * 0.3,
             B=rng.normal(size=(T, G, K)), C=rng.normal(size=(T, G, K)), D=rng.normal(size=C), dt_bias=rng.normal(size=C) * 0.1,
             init_state=rng.normal(size=(3, C, K)))
    if gate:
        a["z"] = rng.normal(size=(T, C))
    dy, dT = rng.normal(size=(T, C)), rng.normal(size=(3, C, K))

    def loss(**v):
        y, fin = S.selective_scan(cu=cu, dt_softplus=softplus, **v)
        return (y * dy).sum() + (fin * dT).sum()

    g = S.selective_scan_bwd(cu=cu, d_out=dy, d_final_state=dT, dt_softplus=softplus, **a)
    names = {"x": "dx", "dt": "ddt", "A_log": "dA_log", "B": "dB", "C": "dC", "D": "dD", "dt_bias": "ddt_bias",
             "init_state": "d_init_state", "z": "dz"}
    differences(loss, a, list(a), {k: g[names[k]] for k in a}, rng)


@pytest.mark.parametrize("activation", [True, False])
def test_conv_gradient_is_the_difference(activation):
    rng = np.random.default_rng(2)
    T, C, W, cu = 8, 3, 4, [0, 2, 2, 8]
    a = dict(x=rng.normal(size=(T, C)), w=rng.normal(size=(C, W)), bias=rng.normal(size=C), conv_state=rng.normal(size=(3, W - 1, C)))
    dy, dT = rng.normal(size=(T, C)), rng.normal(size=(3, W - 1, C))

    def loss(**v):
        y, fin = L.causal_conv1d(cu_seqlens=cu, activation=activation, **v)
        return (y * dy).sum() + (fin * dT).sum()

    g = L.causal_conv1d_bwd(a["x"], a["w"], cu, dy, bias=a["bias"], init_state=a["conv_state"], d_final_state=dT, activation=activation)
    differences(loss, a, list(a), dict(x=g["dx"], w=g["dweight"], bias=g["dbias"], conv_state=g["d_init_state"]), rng)


def test_rotation_by_hand():
    # a quarter turn sends (u, v) to (-v, u); values behind the rotated ones stay
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    c, s = np.zeros((1, 2)), np.ones((1, 2))
    n = x / np.sqrt(np.mean(x * x))
    assert np.allclose(L.norm_rope(x, None, c, s, eps=0.0)[0, 0] * np.sqrt(np.mean(x * x)), [-3, -4, 1, 2, 5, 6])
    assert np.allclose(L.norm_rope(x, None, c, s, eps=0.0, interleaved=True)[0, 0] / n[0, 0, 0], [-2, 1, -4, 3, 5, 6])
    assert np.allclose(np.linalg.norm(L.norm_rope(x, None, c, s, norm="l2", eps=0.0)), 1.0)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_gradient_is_the_difference(norm, interleaved):
    rng = np.random.default_rng(3)
    a = dict(x=rng.normal(size=(3, 2, 8)), weight=1 + 0.1 * rng.normal(size=8))
    th = rng.normal(size=(3, 3))
    c, s, do = np.cos(th), np.sin(th), rng.normal(size=(3, 2, 8))
    kw = dict(norm=norm, eps=1e-3, interleaved=interleaved)
    dx, dw = L.norm_rope_bwd(a["x"], a["weight"], c, s, do, **kw)
    differences(lambda x, weight: (L.norm_rope(x, weight, c, s, **kw) * do).sum(), a, list(a), dict(x=dx, weight=dw), rng)
