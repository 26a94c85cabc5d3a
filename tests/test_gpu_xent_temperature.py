"""Cross entropy where a logit is -inf in fp32 (a product that leaves its range
downwards), at inverse temperatures whose fp32 pair has parts of both signs or
at the end of the range: probability 0 for that entry, and nothing else changes.

The head's residual alone, whole hidden states in one column: the other logits
are q4 2^118 exactly, z between -10 and 10 after scaling.  Exponents are off by two
roundings of z, 2^-23 of 10 each, or by the pair's 2^-23 of twice that: 2^-18 of a
probability, with the exponential's 2^-22 and the sums.  dH has operands and
residual rounded to fp16, 2^-10 of its terms, fp32 sums, 2^-16, and bf16's 2^-8.
"""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


def _head(seed, V, below):
    """Logits of q4 2^118, and of -2^129 at the entries `below`."""
    h = synth.draw_head(np.random.default_rng(seed), V, 256, 0, 0, 64)
    h.c8[...] = 1
    h.s_R[...] = 2.0 ** -9
    h.q4[...] = np.clip(h.q4, -7, 7)
    h.q4[below] = -8
    h.c8[below] = 255
    return h, ah_mod().PackedHead.from_components(h)


def _run(h, head, N, labels, tau, below):
    torch, ah = torch_mod(), ah_mod()
    H = np.zeros((N, 256))
    H[:, 0] = 2.0 ** 127
    tau = float(np.float32(tau * 2.0 ** -118))
    w = np.full(N, 2.0 ** 100)
    dev = lambda x, t: torch.from_numpy(np.asarray(x)).cuda().to(t)  # noqa: E731
    X = dev(H, torch.bfloat16)
    if N <= 32:
        assert torch.isneginf(ah.logits(X, head)[:, below]).all()
    got = ah.archead_cross_entropy(X, dev(labels, torch.int32), head, weight=dev(w, torch.float32), inv_temperature=tau)
    want = oracle.cross_entropy(H, labels, h, w, tau)
    q = -np.expm1(want["logp"])
    err = np.abs(got["logp"].double().cpu().numpy() - want["logp"])
    assert (err <= q * 2.0 ** -18 + 2.0 ** -24 * np.abs(want["logp"])).all(), got["logp"][:4]
    W = np.abs(oracle.w_hat(h))
    z = H @ oracle.w_hat(h).T * tau
    z[np.arange(N), labels] = -np.inf
    e = np.exp(z - z.max(1, keepdims=True))
    T = (w * tau * q)[:, None] * (e / e.sum(1, keepdims=True) @ W + W[labels])
    tol = (2.0 ** -10 + 2.0 ** -16) * T
    tol = tol + 2.0 ** -8 * (np.abs(want["dH"]) + tol) + 2.0 ** -134
    assert (np.abs(got["dH"].double().cpu().numpy() - want["dH"]) <= tol).all()


@pytest.mark.parametrize("tau", [1.0, 0.8, 0.9, 1.25, 0.7, 1.1, 1.3])
@pytest.mark.parametrize("N", [1, 20, 40, 200])
def test_a_logit_below_the_range(N, tau):
    log(f"xent -inf N={N} tau={tau}")
    h, head = _head(N, 500, [77])
    _run(h, head, N, np.random.default_rng(N).integers(78, 500, N), tau, [77])


@pytest.mark.parametrize("N", [1, 20, 40, 200])
def test_runs_of_the_vocabulary_below_the_range(N):
    """Thousands of entries one after the other, and all but the labels' kind."""
    log(f"xent -inf runs N={N}")
    V = 5000
    for first, end in ((0, 2048), (2040, 4200), (4096, 5000)):
        below = np.arange(first, end)
        h, head = _head(N, V, below)
        free = np.setdiff1d(np.arange(V), below)
        _run(h, head, N, np.random.default_rng(N).choice(free, N), 1.25, below)
    below = np.setdiff1d(np.arange(V), [4100])
    h, head = _head(N, V, below)
    _run(h, head, N, np.full(N, 4100), 1.25, below)


@pytest.mark.parametrize("N", [1, 20])
def test_the_ends_of_the_inverse_temperatures_range(N):
    """The largest and the smallest that fp32 holds: equal logits share the
    probability, others have none or all differ by nothing."""
    torch, ah = torch_mod(), ah_mod()
    h, head = _head(N, 500, [77])
    H = torch.zeros((N, 256), device="cuda")
    H[:, 0] = 2.0 ** -60
    lab = torch.full((N,), int(np.flatnonzero(h.q4[:, 0] == h.q4[78:, 0].max())[-1]), dtype=torch.int32, device="cuda")
    top = (h.q4[:, 0] == h.q4[78:, 0].max()).sum()
    for tau, others in ((3.4e38, top), (1e-45, 500)):
        got = ah.archead_cross_entropy(H.bfloat16(), lab, head, inv_temperature=tau)
        assert (got["logp"] + float(np.log(others))).abs().max() <= 2.0 ** -18, (tau, got["logp"][:2])
        assert torch.isfinite(got["dH"]).all()
