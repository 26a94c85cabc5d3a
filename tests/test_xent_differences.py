"""The gradient of the cross entropy against differences of its own loss, with
steps that can tell a wrong gradient from a right one.

Hidden states are whole multiples of 2^-5 below 4, so that a step of 2^-5 either
way is exact in bf16; each row's step is 2^-5 along the signs of its gradient in
the 32 columns where that is largest.  The difference of the two losses is
2 dH.step but for terms of third order in the step; how much those are is taken
from the definition in fp64 at the same three points.
To that come the losses' own errors, q (2 eps + 2^-18) + 2^-24 |log p| each as in
test_gpu_xent.py, and the gradient's, 2^-8 + 2^-10 of its terms along the step.

On the CPU the same test is run on the oracle's loss, and the oracle's gradient
times 0, 1/2, 3/2 and -1 has to fail it.
"""
import numpy as np
import pytest

import oracle
import synth

STEP = 2.0 ** -5
COLUMNS = 32
WRONG = (0.0, 0.5, 1.5, -1.0)


def _case(seed, N, V=800, D=256):
    rng = np.random.default_rng(seed)
    h = synth.draw_head(rng, V, D, 8, 8, 64)
    W = oracle.w_hat(h)
    f = 2.0 / np.sqrt((W ** 2).sum(1).mean())
    for s in (h.s_R, h.s_Ac, h.s_Aw):
        s[...] = (s.astype(np.float64) * f).astype(np.float16)
    H = np.clip(np.round(rng.normal(0, 1, (N, D)) / STEP), -100, 100) * STEP
    return h, oracle.w_hat(h), H, rng.integers(0, V, N)


def _magnitudes(h):
    out = np.abs(h.q4.astype(np.float64)) * np.repeat(h.c8.astype(np.float64), h.g, 1) * np.abs(h.s_R.astype(np.float64))[:, None]
    for A, s_A, B, s_B in ((h.A_c, h.s_Ac, h.B_c, h.s_Bc), (h.A_w, h.s_Aw, h.B_w, h.s_Bw)):
        out += (np.abs(A.astype(np.float64)) * np.abs(s_A.astype(np.float64))[:, None]) @ (
            np.abs(B.astype(np.float64)) * np.repeat(np.abs(s_B.astype(np.float64)), h.g, 1))
    return out


def _steps(dH):
    """Per row +-STEP along the gradient's signs in its largest columns."""
    move = np.zeros_like(dH)
    at = np.argsort(-np.abs(dH), 1)[:, :COLUMNS]
    np.put_along_axis(move, at, STEP * np.sign(np.take_along_axis(dH, at, 1)), 1)
    return move


def _margins(h, W, H, labels, move):
    """Per row, without the gradient's own error, how far the difference of two
    losses may be from 2 dH.step; and the gradient's terms along the step."""
    f = {k: oracle.cross_entropy(H + k * move, labels, h, W=W) for k in (-1, 0, 1)}
    third = f[-1]["logp"] - f[1]["logp"] - 2 * (f[0]["dH"] * move).sum(1)
    Wabs, r = _magnitudes(h), 16
    eps = (H.shape[1] / 16 + r / 16 + 32) * 2.0 ** -24 * ((np.abs(H) + STEP) @ Wabs.T).max(1)
    noise = 2 * (2 * eps + 2.0 ** -18 + 2.0 ** -24 * (np.abs(f[0]["logp"]) + 1))
    z = H @ W.T
    p = np.exp(z - z.max(1, keepdims=True))
    terms = ((p / p.sum(1, keepdims=True) @ Wabs + Wabs[labels]) * np.abs(move)).sum(1)
    return np.abs(third) + noise, terms


def _passes(difference, dH, move, margin, terms):
    own = 2 * (2.0 ** -8 * (np.abs(dH) * np.abs(move)).sum(1) + 2.0 ** -10 * terms)
    return np.abs(difference - 2 * (dH * move).sum(1)) <= margin + own


def test_the_oracle_passes_and_wrong_gradients_do_not():
    for seed in range(5):
        h, W, H, labels = _case(seed, 90)
        dH = oracle.cross_entropy(H, labels, h, W=W)["dH"]
        move = _steps(dH)
        margin, terms = _margins(h, W, H, labels, move)
        up, down = (-oracle.cross_entropy(x, labels, h, W=W)["logp"] for x in (H + move, H - move))
        assert _passes(up - down, dH, move, margin, terms).all()
        for factor in WRONG:
            assert not _passes(up - down, factor * dH, move, margin, terms).any(), (seed, factor)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 32, 90, 300])
def test_gradient_against_differences_of_the_loss(N):
    from tests.gpu_helpers import ah_mod, torch_mod
    torch, ah = torch_mod(), ah_mod()
    for seed in range(3):
        h, W, H, labels = _case(100 + seed, N)
        head = ah.PackedHead.from_components(h)
        lab = torch.from_numpy(labels).int().cuda()

        def call(x):
            t = torch.from_numpy(x).cuda().bfloat16()
            assert np.array_equal(t.double().cpu().numpy(), x)
            return {k: v.double().cpu().numpy() for k, v in ah.archead_cross_entropy(t, lab, head).items()}

        dH = call(H)["dH"]
        move = _steps(dH)
        margin, terms = _margins(h, W, H, labels, move)
        difference = call(H - move)["logp"] - call(H + move)["logp"]
        assert _passes(difference, dH, move, margin, terms).all()
        for factor in WRONG:
            assert not _passes(difference, factor * dH, move, margin, terms).any(), (seed, factor)
