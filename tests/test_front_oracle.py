"""Pins of the oracle in front of the head: the norm's codes by whole-number
arithmetic, its gradient and the cross entropy's against differences, closed
forms."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
import synth


def _bf16(rng, *shape, sigma=1.0):
    return oracle.round_bf16(rng.normal(0, sigma, shape))


def test_round_bf16():
    x = np.array([1.0, 1.00390625, 1.01171875, -3.3e38, 1e-41, np.inf, -np.inf, np.nan])
    got = oracle.round_bf16(x)
    assert got[0] == 1.0 and got[1] == 1.0 and got[2] == 1.015625  # ties to even, down and up
    assert np.isfinite(got[3]) and got[5] == np.inf and got[6] == -np.inf and np.isnan(got[7])
    assert oracle.round_bf16(np.array([3.4e38]))[0] == np.inf
    bits = synth.f32_to_bf16_bits(np.random.default_rng(0).normal(0, 1, 1000).astype(np.float32))
    assert np.array_equal(oracle.bf16_bits_to_f64(bits), oracle.round_bf16(np.random.default_rng(0).normal(0, 1, 1000)))


def _round_half_even(q):
    f = q.numerator // q.denominator
    r = q - f
    return f + (r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2 == 1))


def test_codes_are_the_exact_quotients_rounding():
    """rint(127 t / m) by rational numbers, also with fp32 quotients: the
    border between two codes is never reached by rounding alone."""
    rng = np.random.default_rng(1)
    x, w = _bf16(rng, 40, 61), _bf16(rng, 61)
    x[:, :20] = oracle.round_bf16(x[:, 20:40] * 0.5)  # halves of other columns: exact ties occur
    w[:20] = w[20:40]
    x[7] = 0
    got = oracle.rmsnorm(x, weight=w)
    t = x * w
    m = np.abs(t).max(1)
    for n in range(40):
        want = [0 if m[n] == 0 else _round_half_even(127 * Fraction(v) / Fraction(m[n])) for v in t[n]]
        assert got["codes"][n].tolist() == want
        if m[n]:
            q32 = np.rint((np.float32(127) * t[n].astype(np.float32)) / np.float32(m[n]))
            assert q32.tolist() == want
    assert got["scale"][7] == 0 and abs(got["codes"]).max() == 127
    assert np.allclose(got["codes"] * got["scale"][:, None], got["h"], atol=got["scale"].max() * 0.5001)


def test_norm_closed_form_and_bad_rows():
    x = np.array([[3.0, -4.0], [0.0, 0.0], [np.inf, 1.0], [np.nan, 1.0]])
    got = oracle.rmsnorm(x, weight=np.array([1.0, 2.0]), eps=1e-300)
    assert np.allclose(got["h"][0], [3 / np.sqrt(12.5), -8 / np.sqrt(12.5)])
    assert got["codes"][0].tolist() == [48, -127]  # 127 * 3 / 8 = 47.6
    assert np.isnan(got["scale"][2:]).all() and not got["codes"][1:].any()


@pytest.mark.parametrize("through", [False, True])
def test_norm_gradient_against_differences(through):
    rng = np.random.default_rng(2)
    N, D, eps = 3, 7, 0.01
    x, w, dh, ds = (rng.normal(0, 1, s) for s in ((N, D), D, (N, D), (N, D)))

    def f(x, w):
        return (oracle.rmsnorm(x, weight=w, eps=eps)["h"] * dh).sum() + (ds * x).sum() * through

    got = oracle.rmsnorm_backward(dh, x, oracle.rmsnorm(x, weight=w, eps=eps)["inv_rms"], w, ds if through else None)
    step = 1e-6
    for g, v, call in ((got["dx"], x, lambda u: f(u, w)), (got["dweight"], w, lambda u: f(x, u))):
        for i in np.ndindex(*v.shape):
            up, down = v.copy(), v.copy()
            up[i] += step
            down[i] -= step
            assert abs(g[i] - (call(up) - call(down)) / (2 * step)) < 1e-8


def test_int8_product_is_the_dequantised_one():
    rng = np.random.default_rng(3)
    h = synth.draw_alt_head(rng, 2, 50, 128, 64)
    X, s = rng.integers(-128, 128, (5, 128)), rng.random(5)
    want = np.array([[sum(int(a) * int(b) for a, b in zip(X[n], h.codes[v])) * float(h.scales[v]) * s[n]
                      for v in range(50)] for n in range(5)])
    assert np.allclose(oracle.logits_int8(X, s, h), want, rtol=1e-13)


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_cross_entropy_gradient_against_differences(tau):
    rng = np.random.default_rng(4)
    N, V, D = 5, 21, 128
    head = synth.draw_head(rng, V, D, 8, 8, 64)
    W = oracle.w_hat(head) * 0.05
    H = rng.normal(0, 0.3, (N, D))
    labels, w = rng.integers(0, V, N), np.array([0.2, 0.0, 1.5, -0.3, 0.2])
    got = oracle.cross_entropy(H, labels, head, w, tau, W=W)
    z = H @ W.T * tau
    lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    assert np.allclose(got["logp"][w != 0], lp[np.arange(N), labels][w != 0]) and got["logp"][1] == 0
    assert np.isclose(got["loss"], -(w * got["logp"]).sum()) and not got["dH"][1].any()
    for n in range(N):
        for d in range(0, D, 17):
            up, down = H.copy(), H.copy()
            up[n, d] += 1e-5
            down[n, d] -= 1e-5
            diff = (oracle.cross_entropy(up, labels, head, w, tau, W=W)["loss"]
                    - oracle.cross_entropy(down, labels, head, w, tau, W=W)["loss"]) / 2e-5
            assert abs(got["dH"][n, d] - diff) < 1e-8


def test_cross_entropy_of_a_sure_row_and_of_bad_rows():
    rng = np.random.default_rng(5)
    V, D = 9, 128
    head = synth.draw_head(rng, V, D, 0, 0, 64)
    W = np.eye(V, D)
    H = np.zeros((4, D))
    H[0, 2] = 60.0  # 1 - p = 8 exp(-60): below the last digit of p, not of its gradient
    H[1, 1] = np.nan
    labels = np.array([2, 0, V, 1])
    got = oracle.cross_entropy(H, labels, head, W=W)
    assert np.isclose(got["logp"][0], -8 * np.exp(-60.0), rtol=1e-12)
    assert np.isclose(got["dH"][0, 2], -8 * np.exp(-60.0), rtol=1e-12)
    assert np.isnan(got["logp"][1:3]).all() and np.isnan(got["dH"][1:3]).all() and np.isnan(got["loss"])
    assert np.isclose(got["logp"][3], -np.log(9.0))
    one = synth.draw_head(rng, 1, D, 0, 0, 64)
    got = oracle.cross_entropy(H[:1], [0], one)
    assert got["logp"][0] == 0 and not got["dH"].any()
