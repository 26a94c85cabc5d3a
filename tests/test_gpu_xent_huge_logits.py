"""Cross entropy of logits whose scaled size leaves fp32's whole numbers.

A head of few different rows, each held many times, whole hidden states and
power-of-two scales: logits y are exact in fp32, in any order of their sums, and
equal ones stay equal once they are scaled.  Different ones are 2^-4 apart at
least and inv_temperature is 10^5 and more, or they are 2^18 apart, so that every
probability is 0 or one over the number of entries that share the maximum, to far
below fp64.  The answer follows from counting.

Tolerances.  The entries that share the maximum have equal exponentials, whose
sum is in fp32 runs of 32 (and 2^x by the hardware, 2^-22): 2^-18 of a
probability covers both.  Of rows whose label is below the maximum log p is
z_l - max z, both products of exact numbers with log2(e) inv_temperature: fp64 up
to 32 rows, else two roundings, 2^-23 of z each: 2^-21 of the largest |z| allowed.
dH has operands rounded to fp16 (2^-11) and the residual's (exact here, powers of
two times whole numbers below 8), sums over the vocabulary of V / 16 + 128 fp32
terms, 2^-10 + 2^-16 of the terms in all, and bf16's 2^-8.
"""
import numpy as np
import pytest

import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu

KINDS = 50  # different rows of W; kind k + 25 has the logits of kind k and other columns behind


def _case(seed, N, V, D, exponent):
    rng = np.random.default_rng(seed)
    base = rng.integers(-8, 8, (KINDS, D))
    base[25:, :D - 64] = base[:25, :D - 64]
    # the first half of the vocabulary lacks half of the kinds: maxima rise later on
    kind = np.concatenate([rng.integers(0, 12, V // 2), rng.integers(0, KINDS, V - V // 2)])
    h = synth.draw_head(rng, V, D, 0, 0, 64)
    h.q4[...] = base[kind]
    h.c8[...] = 1
    h.s_R[...] = 2.0 ** -4
    H = rng.integers(-4, 5, (N, D)).astype(np.float64)
    H[:, D - 64:] = 0
    H[0] = 0  # a row of zeros: all entries alike
    H *= 2.0 ** exponent
    return h, base * 2.0 ** -4, kind, H, rng.integers(0, V, N), rng


def _expect(W, kind, H, labels, tau):
    """log p, the rows' (1 - p) and the others' mean row, from counts."""
    y = H @ W.T  # exact
    count = np.bincount(kind, minlength=len(W)).astype(np.float64)
    of = kind[labels]
    others = count - (np.arange(len(W)) == of[:, None])
    top = np.where(others > 0, y, -np.inf).max(1)
    at_top = others * (y == top[:, None])
    k = at_top.sum(1)
    yl = y[np.arange(len(y)), of]
    d = np.log(k) + tau * (top - yl)
    with np.errstate(over="ignore"):
        logp, q = -np.logaddexp(0.0, d), np.exp(-np.logaddexp(0.0, -d))
    return y, logp, q, at_top / k[:, None], of


def _run(N, V, D, tau, exponent, w):
    torch, ah = torch_mod(), ah_mod()
    h, W, kind, H, labels, rng = _case(N + V, N, V, D, exponent)
    head = ah.PackedHead.from_components(h)
    dev = lambda x, t: torch.from_numpy(np.asarray(x)).cuda().to(t)  # noqa: E731
    weight = np.where(rng.random(N) < 0.8, w, 0.0)
    weight[0] = w
    got = ah.archead_cross_entropy(dev(H.astype(np.float32), torch.bfloat16), dev(labels, torch.int32), head,
                                   weight=dev(weight, torch.float32), inv_temperature=tau)
    tau = float(np.float32(tau))
    y, logp, q, mean, of = _expect(W, kind, H, labels, tau)
    on = weight != 0
    logp_got, dH = got["logp"].double().cpu().numpy(), got["dH"].double().cpu().numpy()
    assert not logp_got[~on].any() and not dH[~on].any()
    z = tau * np.abs(y).max(1)
    tol = q * 2.0 ** -18 + 2.0 ** -24 * np.abs(logp) + np.where(np.abs(logp) > 40, 2.0 ** -21 * z, 0)
    err = np.abs(logp_got - logp)
    assert (err <= tol)[on].all(), (logp_got[on][:8], logp[on][:8])
    loss = -(weight * logp).sum()
    assert abs(got["loss"].item() - loss) <= (np.abs(weight) * tol).sum() + 2.0 ** -23 * abs(loss)
    want = (weight * tau * q)[:, None] * (mean @ W - W[of])
    T = (np.abs(weight) * tau * q)[:, None] * (mean @ np.abs(W) + np.abs(W[of]))
    tol = (2.0 ** -10 + 2.0 ** -16 + (V / 16 + 128) * 2.0 ** -24) * T
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134
    assert (np.abs(dH - want) <= tol)[on].all()
    log(f"  N={N} tau={tau} 2^{exponent}: shared maxima {(q[on] > 0).mean():.2f} of the rows")


# log2(e) inv_temperature times the largest logit from 2^22 to 2^31, across the whole range, and by
# the logits' own size
SCALES = [(1e5, 0), (6e5, 0), (1e6, 0), (2.0 ** 20, 0), (3e6, 0), (1e7, 0), (1e8, 0), (1.0, 22), (0.7, 26), (1e30, 0),
          (3e38, -60), (2e-20, 90)]


@pytest.mark.parametrize("tau,exponent", SCALES)
@pytest.mark.parametrize("N", [4, 32, 40, 200])
def test_huge_scaled_logits(N, tau, exponent):
    _run(N, 1003, 256, tau, exponent, 1.0 if tau < 1e20 else 2.0 ** -60)


@pytest.mark.parametrize("tau", [1e6, 1e8])
def test_huge_scaled_logits_in_pieces_of_the_vocabulary(tau):
    _run(2100, 70001, 128, tau, 0, 1.0)


def test_scaled_logits_past_the_range_of_fp32():
    """Up to 32 rows differences are scaled, else the logits: rows in which a
    scaled logit is infinite are NaN then, and no other row is."""
    torch, ah = torch_mod(), ah_mod()
    h, W, kind, H, labels, _ = _case(1, 40, 1003, 256, 0)
    head = ah.PackedHead.from_components(h)
    H[::2] *= 2.0 ** -20
    lab = torch.from_numpy(labels).int().cuda()
    X = torch.from_numpy(H).cuda().bfloat16()
    many = ah.archead_cross_entropy(X, lab, head, weight=torch.full((40,), 2.0 ** -60, device="cuda"), inv_temperature=3e38)
    few = ah.archead_cross_entropy(X[:32], lab[:32], head, weight=torch.full((32,), 2.0 ** -60, device="cuda"),
                                   inv_temperature=3e38)
    bad = torch.arange(40, device="cuda") % 2 == 1
    assert torch.isnan(many["logp"][bad]).all() and torch.isnan(many["dH"][bad]).all()
    assert not torch.isnan(many["logp"][~bad]).any() and not torch.isnan(many["dH"][~bad]).any()
    assert not torch.isnan(few["logp"]).any() and not torch.isnan(few["dH"]).any()
