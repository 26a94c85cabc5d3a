"""Pins of the training oracle: gradients against central differences, closed
forms, and rows that do not count."""
import numpy as np
import pytest

import oracle
import synth


def _difference(f, Y, step=1e-5):
    g = np.zeros(Y.shape)
    for i in np.ndindex(*Y.shape):
        up, down = Y.copy(), Y.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


@pytest.mark.parametrize("s,kl", [(1.0, 0.0), (0.7, 0.1), (1.6, 0.5)])
def test_policy_gradient_against_differences(s, kl):
    rng = np.random.default_rng(int(10 * s))
    N, V = 6, 9
    Y, labels = rng.normal(0, 2, (N, V)), rng.integers(0, V, N)
    base = oracle.policy_loss(Y, labels, np.ones(N), inv_temperature=s)["logp"]
    old = base - np.array([0.05, -0.1, 0.6, 0.6, -0.7, -0.7])  # two kept, then each side of the clip
    args = dict(advantage=np.array([1.0, -0.5, 1.0, -1.0, 1.0, -1.0]), old_logp=old, ref_logp=base + 0.3, kl_coef=kl,
                weight=np.array([1.0, 0.5, 2.0, 0.25, 0.0, 1.0]), inv_temperature=s)
    got = oracle.policy_loss(Y, labels, **args)
    diff = _difference(lambda x: oracle.policy_loss(x, labels, **args)["loss"], Y)
    assert np.allclose(got["dY"], diff, rtol=0, atol=1e-8)
    assert not got["dY"][4].any() and got["logp"][4] == 0
    if kl == 0.0:  # a rise past the clip with a gain, a fall below it with a loss: flat
        assert not got["dY"][2].any() and not got["dY"][5].any() and got["dY"][3].any()


def test_policy_closed_forms():
    Y, labels, A = np.zeros((2, 4)), np.array([1, 3]), np.array([2.0, -3.0])
    got = oracle.policy_loss(Y, labels, A)  # ratio 1: the loss is -sum A, the gradient -A (one-hot - 1/4)
    assert got["loss"] == 1.0 and np.allclose(got["logp"], -np.log(4))
    want = -A[:, None] * (np.eye(4)[labels] - 0.25)
    assert np.allclose(got["dY"], want)
    ref = got["logp"] + np.array([0.0, np.log(2.0)])
    kl = oracle.policy_loss(Y, labels, 0 * A, ref_logp=ref, kl_coef=1.0)
    assert np.allclose(kl["row_loss"], [0.0, 2 - np.log(2) - 1])


def test_a_bad_row_is_nan_and_an_uncounted_one_is_nothing():
    Y = np.zeros((5, 3))
    Y[0] = -np.inf
    Y[1, 1] = np.inf
    Y[2, 2] = np.nan
    labels = np.array([0, 0, 0, 3, 1])
    got = oracle.policy_loss(Y, labels, np.ones(5))
    assert np.isnan(got["logp"][:4]).all() and np.isnan(got["dY"][:4]).all() and np.isfinite(got["dY"][4]).all()
    off = oracle.policy_loss(Y, labels, np.ones(5), weight=np.array([0, 0, 0, 0, 1.0]))
    assert off["loss"] == -1 and not off["dY"][:4].any()


@pytest.mark.parametrize("kind,eps", [(oracle.PREF_SIGMOID, 0.0), (oracle.PREF_SIGMOID, 0.2), (oracle.PREF_SQUARED, 0.0)])
def test_preference_gradient_against_differences(kind, eps):
    rng = np.random.default_rng(3)
    N, V = 9, 7
    Y, labels = rng.normal(0, 2, (N, V)), rng.integers(0, V, N)
    args = dict(offsets=np.array([1, 3, 6, 6, 8]), ref_logp=rng.normal(-2, 0.5, N), kind=kind, beta=0.3,
                weight=np.array([1, 1, 0.5, 1, 0, 2, 1, 1, 1.0]), pair_weight=np.array([1.0, 0.5]), label_smoothing=eps,
                inv_temperature=0.9)
    got = oracle.preference_loss(Y, labels, **args)
    diff = _difference(lambda x: oracle.preference_loss(x, labels, **args)["loss"], Y)
    assert np.allclose(got["dY"], diff, rtol=1e-6, atol=1e-7)
    assert not got["dY"][[0, 4, 8]].any() and not got["logp"][[0, 4, 8]].any()
    assert got["chosen_reward"][1] == 0  # the second pair's chosen sequence has no rows


def test_preference_closed_form():
    Y, labels = np.zeros((2, 4)), np.array([0, 1])
    got = oracle.preference_loss(Y, labels, [0, 1, 2], beta=2.0)  # equal sums: log 2
    assert np.isclose(got["loss"], np.log(2)) and np.isclose(got["dY"][0, 0], -2.0 * 0.5 * 0.75)
    assert np.isclose(got["dY"][1, 1], 2.0 * 0.5 * 0.75)


def test_backward_is_the_adjoint_of_the_forward():
    """<dY, H W^T> = <dY W, H>, for random rows of a ragged head."""
    inp = synth.make("tiny", seed=3, V=77, D=256, N=5, r_c=8, r_r=16, g=64, n_outlier=2)
    dY = np.random.default_rng(5).normal(size=(5, 77))
    Y, dH = oracle.logits(inp.H_bits, inp.head), oracle.logits_backward(dY, inp.head, v_chunk=30)
    H = oracle.bf16_bits_to_f64(inp.H_bits)
    assert np.isclose((dY * Y).sum(), (dH * H).sum(), rtol=1e-12)


def test_own_ratio_is_one_where_log_p_is_minus_infinity():
    Y = np.array([[-np.inf, 0.0, 0.0], [np.nan, 0.0, 0.0]])
    got = oracle.policy_loss(Y, np.array([0, 0]), np.array([2.0, 2.0]))
    assert got["logp"][0] == -np.inf and got["row_loss"][0] == -2.0 and np.array_equal(got["dY"][0], [-2.0, 1.0, 1.0])
    assert np.isnan(got["row_loss"][1]) and np.isnan(got["dY"][1]).all()
