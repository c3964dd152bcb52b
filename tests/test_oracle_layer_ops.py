"""Pins of the fp64 oracles of the decayed linear attention, the rotary positions and the norm with
the residual's addition: hand-worked values, closed forms and finite differences."""
import numpy as np
import pytest

import oracle.add_norm as onorm
import oracle.linear_attn as oattn
import oracle.rotary as orot


def test_linear_attn_by_hand():
    """One head, d = 1, decay 1/2: states 2 * 3 = 6, then 6/2 + 1 * 4 = 7, then 7/2 - 1 * 2 = 1.5."""
    g = np.log([0.5])
    q = np.array([1.0, 2.0, 4.0]).reshape(3, 1, 1)
    k = np.array([2.0, 1.0, -1.0]).reshape(3, 1, 1)
    v = np.array([3.0, 4.0, 2.0]).reshape(3, 1, 1)
    y, s = oattn.forward(q, k, v, g, [0, 3], scale=0.5)
    np.testing.assert_allclose(y.ravel(), [3.0, 7.0, 3.0], rtol=1e-15)
    np.testing.assert_allclose(s.ravel(), [1.5], rtol=1e-15)
    y, s = oattn.forward(q, k, v, g, [0, 0, 3], s0=np.array([5.0, 8.0]).reshape(2, 1, 1, 1))
    np.testing.assert_allclose(s.ravel(), [5.0, 1.5 + 8.0 / 8], rtol=1e-15)
    np.testing.assert_allclose(y[0], [[6.0 + 4.0]], rtol=1e-15)


def test_linear_attn_equals_the_masked_product():
    """y = scale (q k^T weighted e^{g (t - s)}, s <= t) v for every document, shared heads included."""
    rng = np.random.default_rng(0)
    cu, H, Hk, d = [0, 4, 4, 11], 4, 2, 5
    q, k, v = rng.standard_normal((11, H, d)), rng.standard_normal((11, Hk, d)), rng.standard_normal((11, Hk, d))
    g = -rng.uniform(0.0, 1.0, H)
    y, _ = oattn.forward(q, k, v, g, cu, scale=0.7)
    doc = np.searchsorted(cu[1:], np.arange(11), side="right")
    for h in range(H):
        t = np.arange(11)
        w = np.where((t[:, None] >= t) & (doc[:, None] == doc), np.exp(g[h] * np.clip(t[:, None] - t, 0, None)), 0.0)
        ref = 0.7 * ((q[:, h] @ k[:, h // 2].T) * w) @ v[:, h // 2]
        np.testing.assert_allclose(y[:, h], ref, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("name", ["q", "k", "v", "s0"])
def test_linear_attn_gradients_against_differences(name):
    rng = np.random.default_rng(1)
    cu, H, Hk, d = [0, 3, 3, 5], 2, 1, 3
    x = dict(q=rng.standard_normal((5, H, d)), k=rng.standard_normal((5, Hk, d)), v=rng.standard_normal((5, Hk, d)),
             s0=rng.standard_normal((3, H, d, d)))
    g = np.array([-0.3, -1.1])
    dy, dsf = rng.standard_normal((5, H, d)), rng.standard_normal((3, H, d, d))

    def loss(**kw):
        a = {**x, **kw}
        y, s = oattn.forward(a["q"], a["k"], a["v"], g, cu, s0=a["s0"], scale=0.4)
        return np.sum(y * dy) + np.sum(s * dsf)

    grad = oattn.backward(x["q"], x["k"], x["v"], g, cu, dy, s0=x["s0"], ds_final=dsf, scale=0.4)["d" + name]
    for i in np.ndindex(*x[name].shape):
        e = np.zeros_like(x[name])
        e[i] = 1e-4
        num = (loss(**{name: x[name] + e}) - loss(**{name: x[name] - e})) / 2e-4
        # the loss is bilinear in every tensor: the central difference has no truncation error,
        # its rounding is 1e-16 * |loss| / 1e-4
        np.testing.assert_allclose(num, grad[i], atol=1e-9)


def test_rotary_by_hand_and_inverse():
    """Quarter and half turns, both layouts; the inverse undoes them; norms grow by the scale alone."""
    f = np.array([np.pi / 2, np.pi])
    x = np.array([1.0, 2.0, 3.0, 4.0, 9.0]).reshape(1, 1, 5)
    np.testing.assert_allclose(orot.rotate(x, [1], f).ravel(), [-3.0, -2.0, 1.0, -4.0, 9.0], atol=1e-14)
    np.testing.assert_allclose(orot.rotate(x, [1], f, interleaved=True).ravel(), [-2.0, 1.0, -3.0, -4.0, 9.0],
                               atol=1e-14)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 3, 12))
    f, p = rng.uniform(0, 1, 4), rng.integers(0, 1000, 6)
    y = orot.rotate(x, p, f, interleaved=True, scale=1.5)
    np.testing.assert_allclose(orot.rotate(y, p, f, interleaved=True, inverse=True, scale=1 / 1.5), x, atol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(y[..., :8]), 1.5 * np.linalg.norm(x[..., :8]), rtol=1e-12)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])


def test_add_norm_by_hand():
    o, h = onorm.forward([[1.0, 2.0]], [[2.0, 2.0]], [0.0, 1.0], eps=0.0)
    np.testing.assert_allclose(h, [[3.0, 4.0]])
    np.testing.assert_allclose(o, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    q, s = onorm.quantise(np.array([[448.0, 1.06, 17.0, 0.0, 0.0, 0.0]]), 3)
    np.testing.assert_allclose(s, [[1.0, 0.0]])
    np.testing.assert_allclose(q, [[448.0, 1.0, 16.0, 0.0, 0.0, 0.0]])  # 17 ties to the even 16


def test_e4m3_against_torch():
    import torch
    x = np.concatenate([np.linspace(-448, 448, 40001), np.linspace(-0.05, 0.05, 20001)]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(onorm.e4m3(x.astype(np.float64)), ref)


@pytest.mark.parametrize("name", ["h", "w"])
def test_add_norm_gradients_against_differences(name):
    rng = np.random.default_rng(3)
    x = dict(h=rng.standard_normal((3, 8)), w=0.3 * rng.standard_normal(8))
    d_o, d_h = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    g = onorm.backward(x["h"], x["w"], d_o, d_h, 1e-3)
    grad = g["dx"] if name == "h" else g["dw"]

    def loss(**kw):
        a = {**x, **kw}
        o, _ = onorm.forward(a["h"], None, a["w"], 1e-3)
        return np.sum(o * d_o) + np.sum(a["h"] * d_h)

    for i in np.ndindex(*x[name].shape):
        e = np.zeros_like(x[name])
        e[i] = 1e-4
        num = (loss(**{name: x[name] + e}) - loss(**{name: x[name] - e})) / 2e-4
        np.testing.assert_allclose(num, grad[i], atol=1e-6)  # third derivatives of order 10 times 1e-8
