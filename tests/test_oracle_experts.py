"""The expert operators' statements: gradients against differences, 8-bit codes, ragged segments."""
import numpy as np
import pytest

from oracle import experts as ex
from oracle import router


def _diff(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_codes():
    v = ex.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and np.isnan(v[0x7F]) and v[0x88] == -(2.0 ** -6)
    assert len(np.unique(v[~np.isnan(v)])) == 253


def test_norm_gradient():
    rs = np.random.RandomState(0)
    s, g, dy, ds = rs.normal(size=(3, 7)), rs.normal(size=7), rs.normal(size=(3, 7)), rs.normal(size=(3, 7))
    eps = 0.1
    rstd = ex.rms_norm(s, g, eps)[1]
    dx, _, dg, _ = ex.rms_norm_grad(s, g, rstd, dy, ds)
    assert np.allclose(dx, _diff(lambda q: (ex.rms_norm(q, g, eps)[0] * dy).sum() + (q * ds).sum(), s), atol=1e-8)
    assert np.allclose(dg, _diff(lambda q: (ex.rms_norm(s, q, eps)[0] * dy).sum(), g), atol=1e-8)


def test_activation_gradient():
    rs = np.random.RandomState(1)
    h, dy = rs.normal(size=(4, 10)) * 3, rs.normal(size=(4, 5))
    assert np.allclose(ex.silu_gate_grad(h, dy), _diff(lambda q: (ex.silu_gate(q) * dy).sum(), h), atol=1e-7)


@pytest.mark.parametrize("align", [1, 4])
def test_a_layer_and_its_gradients(align):
    """Products, activation, products and combination of one small layer, against differences."""
    rs = np.random.RandomState(2)
    T, E, k, H, I = 5, 4, 2, 6, 3
    ids = np.argsort(rs.rand(1, T, E), -1)[..., :k].astype(np.uint8)
    off, order, inv = (a[0] for a in router.expert_order(ids, E, align, T * k + min(E, T * k) * (align - 1)))
    inv = inv.reshape(T, k)
    x, w1, w2 = rs.normal(size=(T, H)), rs.normal(size=(E, 2 * I, H)), rs.normal(size=(E, H, I))
    wt, dout = rs.rand(T, k), rs.normal(size=(T, H))

    def layer(x, w1, w2, wt):
        h, _ = ex.gemm_rows(x, w1, off, order, k)
        z, _ = ex.gemm_rows(ex.silu_gate(h), w2, off)
        return ex.combine(z, inv, wt)[0]
    h, _ = ex.gemm_rows(x, w1, off, order, k)
    a = ex.silu_gate(h)
    z, _ = ex.gemm_rows(a, w2, off)
    dz, dwt, _ = ex.combine_grad(z, inv, wt, dout, len(order))
    da, _ = ex.gemm_rows(dz, w2.transpose(0, 2, 1), off)
    dw2, _ = ex.gemm_weight_grad(dz, a, off)
    dh = ex.silu_gate_grad(h, da)
    dw1, _ = ex.gemm_weight_grad(dh, x, off, order, k)
    dx = ex.combine(ex.gemm_rows(dh, w1.transpose(0, 2, 1), off)[0], inv)[0]
    # by brute force: every token's experts one by one
    y = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[0, t, j]
            y[t] += wt[t, j] * (w2[e] @ ex.silu_gate((w1[e] @ x[t])[None])[0])
    assert np.allclose(layer(x, w1, w2, wt), y)

    def loss(x, w1, w2, wt):
        return (layer(x, w1, w2, wt) * dout).sum()
    assert np.allclose(dx, _diff(lambda q: loss(q, w1, w2, wt), x), atol=1e-6)
    assert np.allclose(dw1, _diff(lambda q: loss(x, q, w2, wt), w1), atol=1e-6)
    assert np.allclose(dw2, _diff(lambda q: loss(x, w1, q, wt), w2), atol=1e-6)
    assert np.allclose(dwt, _diff(lambda q: loss(x, w1, w2, q), wt), atol=1e-6)
