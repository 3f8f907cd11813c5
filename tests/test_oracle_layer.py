"""Pins of the float64 oracle of the operators around the scan (CPU): every
gradient against central differences of the forward, the forward against closed
forms and against the oracle's other functions.

Central differences with step 1e-6 on float64: truncation ~1e-12 times the
third derivative, rounding ~1e-16 |loss| / 1e-6; the bar 1e-6 (1 + |g|) holds
both with a wide margin at these sizes (|loss| below 1e2)."""
import numpy as np
import pytest

import oracle
from oracle import layer

RNG = np.random.default_rng


def central(loss, a, step=1e-6):
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index", "zerosize_ok"])
    for _ in it:
        i = it.multi_index
        keep = a[i]
        a[i] = keep + step
        up = loss()
        a[i] = keep - step
        g[i] = (up - loss()) / (2 * step)
        a[i] = keep
    return g


def near(g, ref):
    np.testing.assert_array_less(np.abs(g - ref), 1e-6 * (1 + np.abs(ref)))


def test_add_norm_closed_forms():
    x = np.full((2, 8), 3.0)
    out, r = layer.add_norm(x, np.ones(8), eps=0.0)
    np.testing.assert_allclose(out, 1.0)          # a constant row normalises to one
    np.testing.assert_array_equal(r, x)
    res = RNG(0).normal(size=(2, 8))
    out, r = layer.add_norm(x, np.ones(8), residual=res, scale=np.zeros(8))
    np.testing.assert_array_equal(r, res)          # scale 0 leaves the residual
    np.testing.assert_allclose((out ** 2).mean(-1), (res ** 2).mean(-1) / ((res ** 2).mean(-1) + 1e-5))


@pytest.mark.parametrize("with_scale", [False, True])
def test_add_norm_gradients(with_scale):
    rng = RNG(1)
    x, res, w = rng.normal(size=(3, 5)), rng.normal(size=(3, 5)), rng.normal(size=5)
    scale = rng.normal(size=5) if with_scale else None
    dout, dres = rng.normal(size=(3, 5)), rng.normal(size=(3, 5))

    def loss():
        out, r = layer.add_norm(x, w, residual=res, scale=scale)
        return (out * dout).sum() + (r * dres).sum()

    g = layer.add_norm_bwd(dout, layer.add_norm(x, w, residual=res, scale=scale)[1], w, dres=dres,
                           scale=scale, x=x)
    near(g["dx"], central(loss, x))
    near(g["dresidual"], central(loss, res))
    near(g["dw"], central(loss, w))
    if with_scale:
        near(g["dscale"], central(loss, scale))


@pytest.mark.parametrize("before", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_norm_gradients(before, groups):
    rng = RNG(2)
    y, z, w, dout = (rng.normal(size=s) for s in ((2, 6), (2, 6), (6,), (2, 6)))
    loss = lambda: (layer.gated_norm(y, z, w, groups, before=before) * dout).sum()  # noqa: E731
    g = layer.gated_norm_bwd(dout, y, z, w, groups, before=before)
    near(g["dy"], central(loss, y))
    near(g["dz"], central(loss, z))
    near(g["dw"], central(loss, w))


def test_gated_norm_groups_are_separate():
    rng = RNG(3)
    y, z, w = rng.normal(size=(2, 8)), rng.normal(size=(2, 8)), rng.normal(size=8)
    whole = layer.gated_norm(y, z, w, groups=2)
    np.testing.assert_allclose(whole[:, :4], layer.gated_norm(y[:, :4], z[:, :4], w[:4]))
    np.testing.assert_allclose(whole[:, 4:], layer.gated_norm(y[:, 4:], z[:, 4:], w[4:]))


@pytest.mark.parametrize("T", [0, 1, 2, 3, 6])
@pytest.mark.parametrize("act", [0, 1])
def test_conv_gradients(T, act):
    rng = RNG(4)
    x, st = rng.normal(size=(2, T, 3)), rng.normal(size=(2, 3, 3))
    w, b = rng.normal(size=(3, 4)), rng.normal(size=3)
    dout, dst = rng.normal(size=(2, T, 3)), rng.normal(size=(2, 3, 3))

    def loss():  # the oracle's forward takes float32: the convolution written out instead
        seq = np.concatenate([st, x], 1)
        v = b + sum(w[:, j] * seq[:, j:j + T] for j in range(4))
        return ((layer.silu(v) if act else v) * dout).sum() + (seq[:, T:] * dst).sum()

    g = layer.conv1d_bwd(x, w, dout, b, st, dst, act=act)
    near(g["dxbc"], central(loss, x))
    near(g["dw"], central(loss, w))
    near(g["dbias"], central(loss, b))
    near(g["dstate_in"], central(loss, st))


def test_conv_gradient_is_the_forwards():
    """<dout, conv1d(x)> is linear in x without the activation: its gradient
    reproduces the C oracle's forward difference exactly."""
    rng = RNG(5)
    f32 = np.float32
    x, st = rng.normal(size=(1, 7, 4)).astype(f32), rng.normal(size=(1, 3, 4)).astype(f32)
    w, dout = rng.normal(size=(4, 4)).astype(f32), rng.normal(size=(1, 7, 4)).astype(f32)
    out, _ = oracle.conv1d(x, w, None, st, act=0)
    g = layer.conv1d_bwd(x, w, dout, None, st, act=0)
    np.testing.assert_allclose((g["dxbc"] * x).sum() + (g["dstate_in"] * st).sum(), (out * dout).sum())


def test_mixer_step_is_conv_step_then_decode_step():
    rng = RNG(6)
    f32 = np.float32
    B, H, P, G, N, n = 4, 4, 3, 2, 8, 6
    Ch = H * P + 2 * G * N
    conv, h = rng.normal(size=(n, 3, Ch)).astype(f32), rng.normal(size=(n, H, P, N)).astype(f32)
    xbc, dt = rng.normal(size=(B, Ch)).astype(f32), rng.normal(size=(B, H)).astype(f32)
    w, bias = rng.normal(size=(Ch, 4)).astype(f32), rng.normal(size=Ch).astype(f32)
    A, D, db = -rng.uniform(1, 4, H).astype(f32), rng.normal(size=H).astype(f32), rng.normal(size=H).astype(f32)
    slots = np.array([4, -1, 0, 4], np.int32)  # padding, and a slot named twice
    y, conv2, h2 = layer.mixer_step(conv, h, xbc, dt, w, A, G, bias, D, db, 1e-3, 0.1, slots)
    for b, s in ((0, 4), (2, 0)):
        cs = conv[s:s + 1].astype(np.float64)
        v, _ = oracle.conv1d(xbc[b:b + 1, None], w, bias, conv[s:s + 1], act=1)
        v = v[0, 0]
        hs = h[s:s + 1].astype(np.float64)
        for hh in range(H):
            g = hh // 2
            step = float(oracle.delta(dt[b, hh], float(db[hh]), 1e-3, 0.1))
            hs[0, hh] = np.exp(float(A[hh]) * step) * hs[0, hh] + step * np.outer(
                v[hh * P:hh * P + P], v[H * P + g * N:H * P + g * N + N])
        np.testing.assert_allclose(h2[s], hs[0], rtol=1e-12)
        np.testing.assert_array_equal(conv2[s], np.concatenate([cs[0, 1:], xbc[b][None]]))
    np.testing.assert_array_equal(y[[1, 3]], 0.0)
    for s in (1, 2, 3, 5):
        np.testing.assert_array_equal(h2[s], h[s])
        np.testing.assert_array_equal(conv2[s], conv[s])
