"""GPU parity of the losses with the fp64 oracle over temperatures.

The kernels hold s log2 e as two fp32 parts.  Rounded to nearest the second
part has either sign, by s; a logit of -inf (and the maximum of no logits at
all, from which every sum starts) meets both parts.

Tolerances as in test_gpu_loss.py, and for the gradient one term that its
narrow rows do not need: an element is c 2^x / S, and the hardware's 2^x is 0
where it would be below 2^-126.  What is lost is less than 2^-126 |c| / S, so
than 2^-126 |c|, with c = weight slope s: more than one 2^-126 where |c| is
above 1, as at s = 10.
"""
import numpy as np
import pytest

import oracle
from tests import test_gpu_loss as base
from tests.gpu_helpers import torch_mod
from tests.test_gpu_loss import (_check_policy, _check_preference, _make_Y, _policy_case, _run_policy, _run_preference)

pytestmark = pytest.mark.gpu

# second parts of s log2 e below zero to nearest: 0.1, 0.8, 0.9, 1.25, 10; above: 0.7, 2
SCALES = [0.1, 0.7, 0.8, 0.9, 1.25, 2.0, 10.0]
# one workgroup; a few long rows; rows cut into pieces; one launch that holds part of a row, chunks past
# its end among them; the same with every chunk in the row
WAYS = [(4, 300), (5, 9001), (40, 5003), (260, 60001), (257, 100003)]
CASES = ([(n, v, s, masked) for n, v in WAYS[:3] for s in SCALES for masked in (False, True)]
         + [(n, v, s, True) for n, v in WAYS[3:] for s in (0.8, 10.0)])


_check_gradient = base._check_gradient


def _check_gradient_but_flushed(dY, want, slope_tol, s, spread, lp_tol, labels, on, logp, bf16):
    """The check of test_gpu_loss.py after what a 2^x of 0 may lose is taken off the difference."""
    n = np.arange(len(want))
    with np.errstate(all="ignore"):
        c = np.nan_to_num(np.abs(want[n, labels] / np.expm1(logp)))
    diff = dY - want
    lost = np.sign(diff) * np.minimum(np.abs(diff), 2.0 ** -126 * c[:, None])
    _check_gradient(dY - lost, want, slope_tol, s, spread, lp_tol, labels, on, logp, bf16)


@pytest.fixture(autouse=True)
def _flushed(monkeypatch):
    monkeypatch.setattr(base, "_check_gradient", _check_gradient_but_flushed)


def _mask(Y, labels):
    """-inf in most of a row, in its first columns, its last ones, and everywhere but at the label."""
    V = Y.shape[1]
    n = np.arange(V)
    for row, keep in ((0, n % 7 == 3), (1, n >= V // 3), (2, n < 2 * V // 3), (3, n < 0)):
        keep = keep.copy()
        keep[labels[row]] = True
        Y[row, torch_mod().as_tensor(~keep, device="cuda")] = -float("inf")


@pytest.mark.parametrize("y", ["bfloat16", "float32"])
@pytest.mark.parametrize("N,V,s,masked", CASES)
def test_policy_of_every_temperature(N, V, s, y, masked):
    torch = torch_mod()
    print(f"policy N={N} V={V} s={s} {y} masked={masked}", flush=True)
    rng = np.random.default_rng(N + V)
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    c = _policy_case(rng, N, V, Y64, float(np.float32(s)))
    if masked:
        _mask(Y, c["labels"])
        Y64 = Y.double().cpu().numpy()
        lp = oracle.policy_loss(Y64, c["labels"], np.ones(N), inv_temperature=float(np.float32(s)))["logp"]
        c["old_logp"], c["ref_logp"] = (lp - 0.1).astype(np.float32), (lp + 0.2).astype(np.float32)
    c["weight"][:4] = 0.5
    got = _run_policy(Y, c["labels"], c["A"], old_logp=c["old_logp"], ref_logp=c["ref_logp"], weight=c["weight"],
                      clip_high=0.28, kl_coef=0.05, inv_temperature=s)
    assert all(np.isfinite(v).all() for v in got.values())
    _check_policy(got, Y64, c["labels"], c["A"].astype(np.float32), s, 0.05, c["weight"], c["old_logp"], c["ref_logp"],
                  y == "bfloat16")
    if V > 50000:  # without a gradient such rows are cut into pieces as the shorter ones
        return
    plain = _run_policy(Y, c["labels"], c["A"], old_logp=c["old_logp"], ref_logp=c["ref_logp"], weight=c["weight"],
                        clip_high=0.28, kl_coef=0.05, inv_temperature=s, with_gradient=False)
    _check_policy(plain, Y64, c["labels"], c["A"].astype(np.float32), s, 0.05, c["weight"], c["old_logp"],
                  c["ref_logp"], y == "bfloat16")


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
@pytest.mark.parametrize("s", SCALES)
@pytest.mark.parametrize("N,V", WAYS[:3])
def test_preference_of_every_temperature(N, V, s, y, masked):
    torch = torch_mod()
    print(f"preference N={N} V={V} s={s} {y} masked={masked}", flush=True)
    rng = np.random.default_rng(N + V)
    Y, _ = _make_Y(rng, N, V, getattr(torch, y))
    labels = rng.integers(0, V, N)
    if masked:
        _mask(Y, labels)
    Y64 = Y.double().cpu().numpy()
    lp = oracle.policy_loss(Y64, labels, np.ones(N), inv_temperature=float(np.float32(s)))["logp"]
    ref = (lp + rng.normal(0, 0.3, N)).astype(np.float32)
    offsets = [0, 2, N] if N < 8 else [1, 7, 20, 29, N]
    for kind in (0, 1):
        args = dict(ref_logp=ref, beta=0.25, inv_temperature=s, kind=kind)
        got = _run_preference(Y, labels, offsets, **args)
        assert all(np.isfinite(v).all() for v in got.values())
        _check_preference(got, Y64, labels, offsets, y == "bfloat16", **args)
        plain = _run_preference(Y, labels, offsets, with_gradient=False, **args)
        assert "dY" not in plain and all(np.array_equal(plain[k], got[k]) for k in plain)


@pytest.mark.parametrize("s", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 1e-30, 3e37, 2.0 ** 127])
@pytest.mark.parametrize("N,V", [(4, 300), (40, 5003), (260, 60001)])
def test_scales_at_the_ends_of_the_range(N, V, s):
    """Far below 1 every finite logit counts alike, far above it only the
    largest does; -inf never does.  log p is exact to fp32's half step there
    (the sums are of zeros and ones, or rounded by the exponent's bits)."""
    torch = torch_mod()
    rng = np.random.default_rng(V)
    Y, _ = _make_Y(rng, N, V, torch.float32)
    Y[:, 5::2] = -float("inf")
    Y[:, 2] = 100.0
    labels = np.full(N, 2)
    got = _run_policy(Y, labels, np.full(N, 0.5), inv_temperature=s)
    count = V - len(range(5, V, 2))
    p = 1 / count if s < 1 else 1.0
    assert np.allclose(got["logp"], np.log(p), rtol=1e-5, atol=0)
    assert np.isfinite(got["dY"]).all() and got["loss"] == -0.5 * N
    assert not got["dY"][:, 5::2].any()
    want = -0.5 * s * (1 - p)
    assert np.allclose(got["dY"][:, 2], want, rtol=1e-5, atol=2.0 ** -148)
    assert np.allclose(got["dY"][:, 0], 0.5 * s * p if s < 1 else 0.0, rtol=1e-5, atol=2.0 ** -126)
