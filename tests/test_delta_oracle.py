"""Pins of the fp64 oracle of the gated delta rule, rotary positions and layer
norm: hand-worked cases, limits in which they are something known, and central
differences of every gradient."""
import numpy as np
import pytest

import oracle
from oracle import delta as od


def rng(seed):
    return np.random.default_rng(seed)


def case(seed, B=2, N=7, Hk=2, H=4, dk=3, dv=5):
    r = rng(seed)
    k = r.standard_normal((B, N, Hk, dk))
    return dict(q=r.standard_normal((B, N, Hk, dk)), k=k / np.linalg.norm(k, axis=-1, keepdims=True),
                v=r.standard_normal((B, N, H, dv)), g=-0.3 * r.random((B, N, H)), beta=r.random((B, N, H)))


def test_two_tokens_by_hand():
    # dk = 2, dv = 1: k_1 = e_0, k_2 = (e_0 + e_1) / sqrt 2, decay 1/2, beta 1 then 1/2
    k = np.array([[1.0, 0.0], [2 ** -0.5, 2 ** -0.5]]).reshape(1, 2, 1, 2)
    q = np.array([[1.0, 1.0], [0.0, 2.0]]).reshape(1, 2, 1, 2)
    v = np.array([3.0, 5.0]).reshape(1, 2, 1, 1)
    g = np.full((1, 2, 1), np.log(0.5))
    beta = np.array([1.0, 0.5]).reshape(1, 2, 1)
    out, S = od.delta_forward(q, k, v, g, beta)
    # token 1: S = (3, 0), o = 3.  token 2: S' = (1.5, 0), S'.k = 1.5 / sqrt 2,
    # u = (5 - 1.5 / sqrt 2) / 2, S = S' + k u, o = 2 S_1
    u = (5 - 1.5 / 2 ** 0.5) / 2
    assert out[0, 0, 0, 0] == pytest.approx(3.0, abs=1e-14)
    assert S[0, 0, 0, 0] == pytest.approx(1.5 + u / 2 ** 0.5, abs=1e-14)
    assert S[0, 0, 1, 0] == pytest.approx(u / 2 ** 0.5, abs=1e-14)
    assert out[0, 1, 0, 0] == pytest.approx(2 * u / 2 ** 0.5, abs=1e-14)


def test_a_full_correction_recalls_the_last_value():
    c = case(3)
    c["beta"][:] = 1.0
    c["q"] = c["k"]          # reading with the key just written gives its value
    out, _ = od.delta_forward(**c)
    np.testing.assert_allclose(out, c["v"], atol=1e-12)


def test_orthogonal_keys_and_fixed_decay_are_retention():
    # keys e_0 .. e_{N-1}: nothing is ever corrected, so u = v and the rule is retention
    N, H, dv = 6, 2, 3
    r = rng(5)
    k = np.broadcast_to(np.eye(N)[None, :, None, :], (1, N, H, N)).copy()
    q, v = r.standard_normal((1, N, H, N)), r.standard_normal((1, N, H, dv))
    gam = [0.9, 0.6]
    g = np.broadcast_to(np.log(gam), (1, N, H)).copy()
    out, S = od.delta_forward(q, k, v, g, np.ones((1, N, H)))
    ref, Sref = oracle.retention_recurrent(q, k, v, gam)
    np.testing.assert_allclose(out, ref, atol=1e-12)
    np.testing.assert_allclose(S, Sref, atol=1e-12)


def test_split_sequence_lengths_and_reset():
    c = case(7)
    s0 = rng(8).standard_normal((2, 4, 3, 5))
    out, S = od.delta_forward(**c, initial_state=s0)
    a, Sa = od.delta_forward(**{n: x[:, :3] for n, x in c.items()}, initial_state=s0)
    b, Sb = od.delta_forward(**{n: x[:, 3:] for n, x in c.items()}, initial_state=Sa)
    np.testing.assert_allclose(np.concatenate([a, b], 1), out, atol=1e-12)
    np.testing.assert_allclose(Sb, S, atol=1e-12)
    lout, lS = od.delta_forward(**c, initial_state=s0, lengths=[3, 0])
    np.testing.assert_allclose(lout[0, :3], a[0], atol=1e-12)
    assert np.all(lout[0, 3:] == 0) and np.all(lout[1] == 0)
    np.testing.assert_allclose(lS[0], Sa[0], atol=1e-12)
    assert np.array_equal(lS[1], s0[1])
    c["g"][:, 4] = -np.inf   # the state is dropped before token 4
    out, S = od.delta_forward(**c, initial_state=s0)
    b, Sb = od.delta_forward(**{n: x[:, 4:] for n, x in c.items()})
    np.testing.assert_allclose(out[:, 4:], b, atol=1e-12)
    np.testing.assert_allclose(S, Sb, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [5, 2]])
def test_backward_against_differences(lengths):
    c = case(11, N=5, dk=2, dv=3)
    r = rng(12)
    s0, dS = r.standard_normal((2, 4, 2, 3)), r.standard_normal((2, 4, 2, 3))
    do = r.standard_normal(c["v"].shape)

    def loss(c, s0):
        out, S = od.delta_forward(**c, initial_state=s0, lengths=lengths)
        return (out * do).sum() + (S * dS).sum()

    grads = od.delta_backward(**c, dout=do, initial_state=s0, dfinal_state=dS, lengths=lengths)
    h = 1e-6
    for name in ("q", "k", "v", "g", "beta", "initial_state"):
        x = s0 if name == "initial_state" else c[name]
        num = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            old = x[i]
            x[i] = old + h
            up = loss(c, s0)
            x[i] = old - h
            num[i] = (up - loss(c, s0)) / (2 * h)
            x[i] = old
        np.testing.assert_allclose(grads["d" + name], num, atol=2e-8)


def test_rotary_layouts_inverse_and_relative_positions():
    r = rng(21)
    x, y = r.standard_normal((2, 3, 2, 8)), r.standard_normal((2, 3, 2, 8))
    f = np.array([0.7, 0.01, 1e-3])  # six of the eight components
    pos = np.array([[0, 5, 7], [100, 3, 40]])
    for layout in ("interleaved", "half"):
        z = od.rotary(x, pos, f, layout)
        np.testing.assert_array_equal(z[..., 6:], x[..., 6:])
        np.testing.assert_allclose(z[0, 0], x[0, 0], atol=1e-15)          # position 0
        np.testing.assert_allclose((z ** 2).sum(-1), (x ** 2).sum(-1))     # a rotation
        np.testing.assert_allclose(od.rotary(z, pos, f, layout, inverse=True), x, atol=1e-14)
        # <R_m x, R_n y> depends on m - n alone
        a = (od.rotary(x, pos + 9, f, layout) * od.rotary(y, pos + 2, f, layout)).sum(-1)
        b = (od.rotary(x, pos + 7, f, layout) * od.rotary(y, pos, f, layout)).sum(-1)
        np.testing.assert_allclose(a, b, atol=1e-12)
    np.testing.assert_allclose(od.rotary(x, pos, f, "half", scale=1.5), 1.5 * od.rotary(x, pos, f, "half") -
                               0.5 * np.concatenate([0 * x[..., :6], x[..., 6:]], -1))
    full = oracle.xpos_rotate(x, 5)  # the library's own rotation is the plain interleaved one
    np.testing.assert_allclose(full, od.rotary(x, np.broadcast_to(5 + np.arange(3), (2, 3)),
                                               10000.0 ** (-np.arange(4) / 4)), atol=1e-12)


def test_layernorm_gradients_against_differences():
    r = rng(31)
    x, dy, gain, bias = (r.standard_normal(s) for s in ((4, 6), (4, 6), (6,), (6,)))
    y, mean, rstd = od.layernorm(x, gain, bias)
    np.testing.assert_allclose(((y - bias) / gain).mean(-1), 0, atol=1e-12)
    dx, dgain, dbias = od.layernorm_backward(dy, x, mean, rstd, gain)
    h = 1e-6
    for a, ref in ((x, dx), (gain, dgain), (bias, dbias)):
        for i in np.ndindex(*a.shape):
            old = a[i]
            a[i] = old + h
            up = (od.layernorm(x, gain, bias)[0] * dy).sum()
            a[i] = old - h
            dn = (od.layernorm(x, gain, bias)[0] * dy).sum()
            a[i] = old
            assert abs((up - dn) / (2 * h) - ref[i]) < 2e-8
