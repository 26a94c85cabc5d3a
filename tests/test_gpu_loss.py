"""GPU parity of the policy and preference losses with the fp64 oracle.

Tolerances, from the kernels' arithmetic (u = 2^-24, half an fp32 step):
  log p   The sum of exponentials S is the only fp32 quantity with more than
          one rounding.  A term 2^x has the exponential's ulp (2u), and the two
          roundings of its argument, 2u |x| ln 2; weighted with the term
          itself, |x| 2^x < 0.54, that adds less than 2u for the terms of a few
          units below the maximum, and 2u x ln 2 at most for x the row's
          spread in octaves (at most 150: lower terms are nothing in fp32).
          Adding: a thread adds at most V / 256 terms (of one piece), each
          addition u.  Merging pieces, waves and lanes: 2u for the rescaling
          and u for the sum, at most 6 + 4 + 64 levels.  Storing rounds by
          u |log p|.
              lp_tol = u (|log p| + 2 spread + V / 256 + 3 * 74 + 4)
  l_n     moves by |dl/dlog p| lp_tol; stored with u |l_n|.  The derivative
          is bounded by r |A| + kl_coef (e^d + 1), times 1.01 for the move.
  sums    the sum over rows of |w| times the rows' errors, then u.
  dY      an element off the label is c 2^x / S: the exponential as above,
          u (2 + 2 |x|), c / S rounded once, a pair's slope and its product
          with c / S once each, the product once, and S's own error
          e_S <= lp_tol:  |dY| (u (8 + 2 spread) + lp_tol);  the label's has
          fewer, and its 1 - p moves by p lp_tol.  All move with the
          coefficient's error, |w| s |d slope| p, where the slope moves by the
          same bound as l_n's.  bf16 adds 2^-8 |dY| and fp32 subnormals may
          flush: 2^-126.
"""
import warnings

import warnings

import numpy as np
import pytest

import oracle
from tests.gpu_helpers import ah_mod, torch_mod

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev(x, dtype=None):
    torch = torch_mod()
    return None if x is None else torch.as_tensor(np.asarray(x), dtype=dtype, device="cuda")


def _f32(x):
    return None if x is None else np.asarray(x, np.float32).astype(np.float64)


def _make_Y(rng, N, V, dtype, pad=0, first=0):
    """(device logits with row stride V + pad starting at element `first`, fp64 copy)."""
    torch = torch_mod()
    buf = torch.full((N * (V + pad) + first,), float("nan"), dtype=dtype, device="cuda")
    Y = buf[first:first + N * (V + pad)].view(N, V + pad)[:, :V]
    Y.copy_(torch.as_tensor(rng.normal(0, 3, (N, V)).astype(np.float32)))
    return Y, Y.double().cpu().numpy()


def _spread(Y64, s):
    fin = np.where(np.isfinite(Y64), Y64, np.nan)
    with np.errstate(all="ignore"), warnings.catch_warnings():
        warnings.simplefilter("ignore", RuntimeWarning)  # rows with nothing finite
        return np.minimum(np.nan_to_num(np.nanmax(fin, 1) - np.nanmin(fin, 1)) * s / np.log(2), 150.0)


def _lp_tol(logp, spread, V):
    return U * (np.abs(logp) + 2 * spread + V / 256 + 3 * 74 + 4)


def _check_rows(got, want, tol, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    ok = ~np.isnan(want)
    worst = np.max((np.abs(got - want) / np.maximum(tol, 1e-300))[ok], initial=0.0)
    print(f"  {what}: worst error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def _check_gradient(dY, want, slope_tol, s, spread, lp_tol, labels, on, logp, bf16):
    """slope_tol: bound of the error of weight x slope, per row."""
    p = np.zeros_like(want)
    rows = np.flatnonzero(on & ~np.isnan(want).any(1))
    with np.errstate(all="ignore"):
        coef = np.zeros(len(want))
        for n in rows:
            q = want[n].copy()
            q[labels[n]] = 0
            denom = -np.expm1(logp[n])
            coef[n] = want[n, labels[n]] / denom if denom != 0 else 0.0
            p[n] = np.abs(q / coef[n]) if coef[n] != 0 else 1.0
            p[n, labels[n]] = 1.0
    rel = U * (8 + 2 * spread) + lp_tol
    tol = np.abs(want) * rel[:, None] + p * (slope_tol * s)[:, None] + np.abs(coef * lp_tol)[:, None] * p + 2.0 ** -126
    if bf16:
        tol = tol * (1 + 2 ** -8) + np.abs(want) * 2.0 ** -8
    _check_rows(dY, want, tol, "dY")


def _run_policy(Y, labels, A, **kw):
    torch = torch_mod()
    f = lambda x: _dev(x, torch.float32)
    kw = dict(kw)
    for k in ("old_logp", "ref_logp", "weight"):
        kw[k] = f(kw.get(k))
    out = ah_mod().archead_policy_loss(Y, _dev(labels, torch.int32), f(A), **kw)
    torch.cuda.synchronize()
    return {k: v.double().cpu().numpy() for k, v in out.items()}


def _policy_case(rng, N, V, Y64, s):
    """Labels, advantages, old and reference log-probabilities away from the
    clip's borders, weights of which some are zero."""
    labels = rng.integers(0, V, N)
    base = oracle.policy_loss(Y64, labels, np.ones(N), inv_temperature=s)["logp"]
    delta = rng.normal(0, 0.3, N)
    for border in (np.log(0.8), np.log(1.28)):
        delta = np.where(np.abs(delta - border) < 1e-3, border + 3e-3, delta)
    w = rng.uniform(0.2, 1.5, N)
    w[rng.random(N) < 0.25] = 0.0
    return dict(labels=labels, A=rng.normal(0.2, 1, N), old_logp=(base - delta).astype(np.float32),
                ref_logp=(base + rng.normal(0, 0.3, N)).astype(np.float32), weight=w.astype(np.float32))


def _check_policy(got, Y64, labels, A, s, kl, weight, old_logp, ref_logp, bf16, clip_low=0.2, clip_high=0.28):
    kw = dict(old_logp=_f32(old_logp), ref_logp=_f32(ref_logp), weight=_f32(weight), clip_low=float(np.float32(clip_low)),
              clip_high=float(np.float32(clip_high)), kl_coef=float(np.float32(kl)), inv_temperature=float(np.float32(s)))
    want = oracle.policy_loss(Y64, labels, _f32(A), **kw)
    V, spread = Y64.shape[1], _spread(Y64, s)
    w = np.ones(len(Y64)) if weight is None else _f32(weight)
    lp_tol = _lp_tol(want["logp"], spread, V)
    _check_rows(got["logp"], want["logp"], lp_tol, "logp")
    with np.errstate(all="ignore"):
        r = 1.0 if old_logp is None else np.exp(want["logp"] - kw["old_logp"])
        e = kl * (np.exp(kw["ref_logp"] - want["logp"]) + 1) if kl else 0.0
        move = np.nan_to_num(1.01 * (r * np.abs(_f32(A)) + e)) * lp_tol
    _check_rows(got["row_loss"], want["row_loss"], move + U * np.abs(want["row_loss"]), "row_loss")
    total = np.sum(np.abs(w) * move) + U * np.abs(want["loss"])
    _check_rows(got["loss"][None], np.array([want["loss"]]), np.array([total]), "loss")
    if "dY" in got:
        _check_gradient(got["dY"], want["dY"], np.abs(w) * move, s, spread, lp_tol, labels, w != 0, want["logp"], bf16)
    return want


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 8), (5, 255), (4, 1024), (7, 2049), (3, 5003), (2, 33001), (1, 151936), (70, 777),
          (300, 130), (600, 33001), (260, 60001)]


@pytest.mark.parametrize("y,dy", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float32", "bfloat16"),
                                  ("bfloat16", "float32")])
@pytest.mark.parametrize("N,V", SHAPES)
def test_policy_matches_oracle(N, V, y, dy):
    torch = torch_mod()
    print(f"policy N={N} V={V} {y} {dy}", flush=True)
    rng = np.random.default_rng(1000 * N + V)
    s, kl = 0.75, 0.05
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    c = _policy_case(rng, N, V, Y64, s)
    got = _run_policy(Y, c["labels"], c["A"], old_logp=c["old_logp"], ref_logp=c["ref_logp"], weight=c["weight"],
                      clip_high=0.28, kl_coef=kl, inv_temperature=s, dY_dtype=getattr(torch, dy))
    assert np.array_equal(Y.double().cpu().numpy(), Y64)
    _check_policy(got, Y64, c["labels"], c["A"].astype(np.float32), s, kl, c["weight"], c["old_logp"], c["ref_logp"],
                  dy == "bfloat16")


def test_policy_plain_forms():
    """No old policy, no reference, no weights, no clip, no gradient."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    Y, Y64 = _make_Y(rng, 6, 3001, torch.float32)
    labels, A = rng.integers(0, 3001, 6), rng.normal(0, 1, 6).astype(np.float32)
    got = _run_policy(Y, labels, A)
    _check_policy(got, Y64, labels, A, 1.0, 0.0, None, None, None, False, 0.2, 0.2)
    old = (got["logp"] + rng.normal(0, 1, 6)).astype(np.float32)
    got = _run_policy(Y, labels, A, old_logp=old, clip_low=float("inf"), clip_high=float("inf"))
    _check_policy(got, Y64, labels, A, 1.0, 0.0, None, old, None, False, float("inf"), float("inf"))
    got = _run_policy(Y, labels, A, with_gradient=False)
    assert "dY" not in got


def test_policy_wide_ratio_and_kl():
    """Log-ratios of many units, both signs of the advantage, zero advantage."""
    torch = torch_mod()
    rng = np.random.default_rng(6)
    N, V = 12, 513
    Y, Y64 = _make_Y(rng, N, V, torch.bfloat16)
    labels = rng.integers(0, V, N)
    base = oracle.policy_loss(Y64, labels, np.ones(N))["logp"]
    old = (base + np.repeat([-6.0, 0.0, 6.0], 4)).astype(np.float32)
    ref = (base + np.tile([-5.0, 5.0], 6)).astype(np.float32)
    A = np.tile([1.5, -1.5, 0.0, 1.0], 3).astype(np.float32)
    for kl in (0.0, 0.3):
        got = _run_policy(Y, labels, A, old_logp=old, ref_logp=ref, kl_coef=kl, clip_high=0.28, dY_dtype=torch.float32)
        _check_policy(got, Y64, labels, A, 1.0, kl, None, old, ref, False)


# columns and copies of the rows below: one workgroup, a few long rows, rows cut into pieces
WAYS = [(1500, 1), (9000, 1), (9000, 3)]


@pytest.mark.parametrize("V,copies", WAYS)
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
def test_policy_uncounted_rows_hold_anything(y, V, copies):
    torch = torch_mod()
    rng = np.random.default_rng(7)
    N = 9 * copies
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    c = _policy_case(rng, N, V, Y64, 1.0)
    w = c["weight"].copy()
    w[:] = 0.5
    w[[0, 3, 8]] = 0
    args = dict(old_logp=c["old_logp"], ref_logp=c["ref_logp"], weight=w, kl_coef=0.05, clip_high=0.28)
    clean = _run_policy(Y, c["labels"], c["A"], **args)
    Y[0] = float("nan")
    Y[3] = float("inf")
    Y[8] = -float("inf")
    labels, old, A = c["labels"].copy(), c["old_logp"].copy(), c["A"].copy()
    labels[[0, 3, 8]] = -100, V, 2 ** 31 - 1
    old[[0, 3]] = np.nan, -np.inf
    A[[3, 8]] = np.nan, np.inf
    got = _run_policy(Y, labels, A, **dict(args, old_logp=old))
    for k in clean:
        assert np.array_equal(got[k], clean[k]), k
    assert not got["dY"][[0, 3, 8]].any() and not got["logp"][[0, 3, 8]].any()
    none = _run_policy(Y, labels, A, **dict(args, old_logp=old, weight=np.zeros(N)))
    assert none["loss"] == 0 and not none["dY"].any() and not none["row_loss"].any()


@pytest.mark.parametrize("V,copies", WAYS)
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
def test_policy_masked_vocabulary(y, V, copies):
    """Logits of -inf and of the type's lowest value in most of a row, whole
    pieces of it among them; rows with nothing left, NaN or +inf are NaN."""
    torch = torch_mod()
    rng = np.random.default_rng(8)
    N, at = 8, V // 2
    Y, _ = _make_Y(rng, N, V, getattr(torch, y))
    labels = np.full(N, at)
    Y[0, :at - 100] = -float("inf")
    Y[1, at + 1:] = -float("inf")
    Y[2, :] = torch.finfo(Y.dtype).min
    Y[3, :at] = torch.finfo(Y.dtype).min
    Y[4] = -float("inf")
    Y[4, at] = 1.0
    Y[5] = -float("inf")
    Y[6, 17] = float("nan")
    Y[7, V - 1] = float("inf")
    Y, labels = Y.repeat(copies, 1), np.tile(labels, copies)
    Y64 = Y.double().cpu().numpy()
    A = np.ones(N * copies, np.float32)
    got = _run_policy(Y, labels, A)
    want = _check_policy(got, Y64, labels, A, 1.0, 0.0, None, None, None, y == "bfloat16", 0.2, 0.2)
    assert np.isnan(got["logp"][5:8]).all() and np.isfinite(got["logp"][:5]).all() and np.isnan(got["loss"])
    assert abs(got["logp"][2] + np.log(V)) < 1e-5 and got["logp"][4] == 0.0 and not got["dY"][4].any()
    assert not got["dY"][0, :at - 100].any() and np.isfinite(want["dY"][:5]).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
def test_policy_many_rows_with_special_ones(y, in_place):
    """Enough rows and columns for the fused kernel: rows that do not count (in
    runs and alone), -inf at the front, in the middle and everywhere, logits far
    above the row's first ones, the type's lowest value, NaN, +inf, labels out
    of range; a stride that is no multiple of 16 bytes."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    N, V = 280, 50003
    Y, _ = _make_Y(rng, N, V, getattr(torch, y), pad=2, first=3)
    w = np.full(N, 0.5)
    w[40:90] = 0
    w[[0, 100, 279]] = 0
    labels = rng.integers(0, V, N)
    labels[:V // 4096] = np.arange(V // 4096) * 4096 + 4095
    labels[20:24] = 0, V - 1, V - 2, V // 8 * 8
    Y[[0, 45, 279]] = float("nan")
    Y[100] = float("inf")
    labels[[0, 45, 100, 279]] = -100
    Y[1, :30000] = -float("inf")       # the first chunks of every thread
    Y[2, :8] = -float("inf")           # ... of one
    Y[3, 8:40000] = -float("inf")
    Y[4] = torch.finfo(Y.dtype).min
    Y[5, :V - 5] = torch.finfo(Y.dtype).min
    Y[6, 40000] = 3000.0               # 2^k times the first chunks' maximum is infinite
    Y[7, 5] = 3000.0
    Y[8] = -2000.0
    labels[1:9] = 40000, 40001, 40002, 3, V - 1, 40000, 17, 0
    Y[9] = -float("inf")
    Y[10, 49999] = float("nan")
    Y[11, 3] = float("inf")
    labels[12:14] = -1, V
    Y64, A = Y.double().cpu().numpy(), rng.normal(0.2, 1, N).astype(np.float32)
    got = _run_policy(Y, labels, A, weight=w, **(dict(dY=Y) if in_place else {}))
    assert np.isnan(got["logp"][9:14]).all() and np.isfinite(got["logp"][:9]).all()
    _check_policy(got, Y64, labels, A, 1.0, 0.0, w, None, None, y == "bfloat16", 0.2, 0.2)
    none = _run_policy(Y, labels, A, weight=0 * w)
    assert none["loss"] == 0 and not none["dY"].any()


def test_policy_label_out_of_range_is_nan():
    torch = torch_mod()
    rng = np.random.default_rng(9)
    Y, Y64 = _make_Y(rng, 4, 100, torch.float32)
    labels, A = np.array([3, -1, 100, 99]), np.ones(4, np.float32)
    got = _run_policy(Y, labels, A)
    _check_policy(got, Y64, labels, A, 1.0, 0.0, None, None, None, False, 0.2, 0.2)
    assert np.array_equal(np.isnan(got["dY"]).all(1), [False, True, True, False])


@pytest.mark.parametrize("V", [1000, 20001])  # one workgroup, a few long rows
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
def test_policy_strides_alignments_and_in_place(y, V):
    """A gradient over its logits, rows of an odd stride and a start off every
    alignment: the same bits as the plain call; nothing beside the rows is written."""
    torch = torch_mod()
    ah = ah_mod()
    rng = np.random.default_rng(V)
    N, dt = 5, getattr(torch, y)
    Y, Y64 = _make_Y(rng, N, V, dt)
    c = _policy_case(rng, N, V, Y64, 1.0)
    f = lambda x: _dev(x, torch.float32)
    args = dict(old_logp=f(c["old_logp"]), ref_logp=f(c["ref_logp"]), weight=f(c["weight"]), kl_coef=0.1)
    labels, A = _dev(c["labels"], torch.int32), f(c["A"])
    base = ah.archead_policy_loss(Y, labels, A, **args)
    for pad, first in ((0, 0), (3, 1), (7, 5)):
        buf = torch.full((N * (V + pad) + first + 9,), 7.0, dtype=dt, device="cuda")
        view = buf[first:first + N * (V + pad)].view(N, V + pad)[:, :V]
        view.copy_(Y)
        got = ah.archead_policy_loss(view, labels, A, dY=view, **args)
        torch.cuda.synchronize()
        assert got["dY"] is view
        for k in base:
            assert torch.equal(got[k], base[k]), (k, pad, first)
        view.fill_(7.0)
        assert (buf == 7.0).all(), "written beside the rows"
        # dY in other rows' padding: Y and dY of different strides
        out = torch.full((N, V + pad + 2), 5.0, dtype=dt, device="cuda")
        got = ah.archead_policy_loss(Y, labels, A, dY=out[:, 1:V + 1], **args)
        torch.cuda.synchronize()
        assert torch.equal(got["dY"], base["dY"]) and (out[:, 0] == 5).all() and (out[:, V + 1:] == 5).all()


def test_losses_are_deterministic_and_empty_calls_are_zero():
    torch = torch_mod()
    ah = ah_mod()
    rng = np.random.default_rng(11)
    Y, _ = _make_Y(rng, 40, 70001, torch.bfloat16)
    labels = _dev(rng.integers(0, 70001, 40), torch.int32)
    A = _dev(rng.normal(0, 1, 40), torch.float32)
    off = _dev([0, 10, 20, 30, 40], torch.int32)
    first = [ah.archead_policy_loss(Y, labels, A), ah.archead_preference_loss(Y, labels, off)]
    for _ in range(3):
        for a, b in zip(first, [ah.archead_policy_loss(Y, labels, A), ah.archead_preference_loss(Y, labels, off)]):
            assert all(torch.equal(a[k], b[k]) for k in a)
    empty = ah.archead_policy_loss(Y[:0], labels[:0], A[:0])
    assert empty["loss"].item() == 0 and empty["dY"].shape == (0, 70001)
    empty = ah.archead_preference_loss(Y[:0], labels[:0], off[:1])
    assert empty["loss"].item() == 0
    # one pair without rows: h = 0
    empty = ah.archead_preference_loss(Y[:0], labels[:0], _dev([0, 0, 0], torch.int32))
    assert abs(empty["loss"].item() - np.log(2)) < 1e-7 and empty["chosen_reward"].item() == 0


# ---------------------------------------------------------------- preference ---

def _run_preference(Y, labels, offsets, **kw):
    torch = torch_mod()
    kw = dict(kw)
    for k in ("ref_logp", "weight", "pair_weight"):
        kw[k] = _dev(kw.get(k), torch.float32)
    out = ah_mod().archead_preference_loss(Y, _dev(labels, torch.int32), _dev(offsets, torch.int32), **kw)
    torch.cuda.synchronize()
    return {k: v.double().cpu().numpy() for k, v in out.items()}


def _check_preference(got, Y64, labels, offsets, bf16, ref_logp=None, weight=None, pair_weight=None, beta=0.1,
                      label_smoothing=0.0, inv_temperature=1.0, kind=0):
    f = lambda x: float(np.float32(x))
    want = oracle.preference_loss(Y64, labels, offsets, ref_logp=_f32(ref_logp), weight=_f32(weight),
                                  pair_weight=_f32(pair_weight), beta=f(beta), label_smoothing=f(label_smoothing),
                                  inv_temperature=f(inv_temperature), kind=kind)
    N, V = Y64.shape
    B, spread = (len(offsets) - 1) // 2, _spread(Y64, inv_temperature)
    w = np.ones(N) if weight is None else _f32(weight)
    pw = np.ones(B) if pair_weight is None else _f32(pair_weight)
    lp_tol = _lp_tol(want["logp"], spread, V)
    _check_rows(got["logp"], want["logp"], lp_tol, "logp")
    off = np.clip(offsets, 0, N)
    # a sequence sum moves by its rows' |w| lp_tol; the loss by its slope's bound times that, the slope by its curvature's
    seq = np.array([np.sum((np.abs(w) * lp_tol)[off[i]:off[i + 1]]) for i in range(2 * B)])
    dh = seq[0::2] + seq[1::2]
    for k, q in (("chosen_reward", seq[0::2]), ("rejected_reward", seq[1::2])):
        _check_rows(got[k], want[k], beta * q + U * np.abs(want[k]), k)
    if kind == 0:
        slope, curve = np.full(B, beta), np.full(B, beta * beta)
    else:
        h = (want["chosen_reward"] - want["rejected_reward"]) / beta
        slope, curve = 2 * np.abs(h - 0.5 / beta) + 2 * dh, np.full(B, 2.0)
    total = np.sum(np.abs(pw) * slope * dh) + U * abs(want["loss"])
    _check_rows(got["loss"][None], np.array([want["loss"]]), np.array([total]), "loss")
    # fp64 slopes: their error is the curvature times dh (and a few fp64 roundings)
    row_tol, on = np.zeros(N), np.zeros(N, bool)
    for i in range(2 * B):
        row_tol[off[i]:off[i + 1]] = np.abs(pw[i // 2]) * (curve[i // 2] * dh[i // 2] + 2.0 ** -40 * slope[i // 2])
        on[off[i]:off[i + 1]] = True
    _check_gradient(got["dY"], want["dY"], np.abs(w) * row_tol, inv_temperature, spread, lp_tol, labels, on & (w != 0),
                    want["logp"], bf16)
    return want


PAIRS = [  # N, V, offsets
    (2, 5, [0, 1, 2]),
    (12, 1000, [0, 5, 12]),
    (40, 2049, [0, 7, 20, 21, 40]),
    (40, 513, [3, 7, 7, 21, 30]),            # an empty sequence, rows before and behind
    (9, 20001, [0, 2, 4, 6, 7, 8, 9]),
    (64, 1000, list(range(0, 65, 2))[:33]),  # sixteen pairs of four rows, one workgroup
    (600, 97, [0, 300, 600]),                # more rows than a workgroup has threads
]


@pytest.mark.parametrize("y,dy", [("bfloat16", "bfloat16"), ("float32", "float32"), ("bfloat16", "float32")])
@pytest.mark.parametrize("kind,eps", [(0, 0.0), (0, 0.1), (1, 0.0)])
@pytest.mark.parametrize("N,V,offsets", PAIRS)
def test_preference_matches_oracle(N, V, offsets, kind, eps, y, dy):
    torch = torch_mod()
    print(f"preference N={N} V={V} offsets={offsets} kind={kind} eps={eps} {y} {dy}", flush=True)
    rng = np.random.default_rng(N + V)
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    labels = rng.integers(0, V, N)
    base = oracle.policy_loss(Y64, labels, np.ones(N), inv_temperature=0.75)["logp"]
    w = rng.uniform(0.5, 1.0, N).astype(np.float32)
    w[rng.random(N) < 0.2] = 0
    args = dict(ref_logp=(base + rng.normal(0, 0.3, N)).astype(np.float32), weight=w,
                pair_weight=rng.uniform(0.2, 1, len(offsets) // 2).astype(np.float32), beta=0.25, label_smoothing=eps,
                inv_temperature=0.75, kind=kind)
    got = _run_preference(Y, labels, offsets, dY_dtype=getattr(torch, dy), **args)
    _check_preference(got, Y64, labels, offsets, dy == "bfloat16", **args)
    got = _run_preference(Y, labels, offsets, beta=0.25, kind=kind)  # reference-free, no weights
    _check_preference(got, Y64, labels, offsets, y == "bfloat16", beta=0.25, kind=kind)


@pytest.mark.parametrize("y,V", [("bfloat16", 40001), ("float32", 20003)])
def test_preference_of_many_long_rows(y, V):
    """Enough work that pieces are whole rounds of a workgroup's loads, which a
    row's last piece is not."""
    torch = torch_mod()
    rng = np.random.default_rng(V)
    N, offsets = 430, [3, 150, 200, 420, 425]
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    labels = rng.integers(0, V, N)
    labels[:4] = V - 1
    got = _run_preference(Y, labels, offsets, beta=0.25)
    _check_preference(got, Y64, labels, offsets, y == "bfloat16", beta=0.25)


def test_preference_large_margins_stay_finite():
    torch = torch_mod()
    rng = np.random.default_rng(2)
    Y, Y64 = _make_Y(rng, 8, 300, torch.float32)
    labels = rng.integers(0, 300, 8)
    for side in (1, -1):
        ref = np.repeat([side * 300.0, -side * 300.0], 4).astype(np.float32)
        got = _run_preference(Y, labels, [0, 4, 8], ref_logp=ref, beta=1.0, label_smoothing=0.1)
        _check_preference(got, Y64, labels, [0, 4, 8], False, ref_logp=ref, beta=1.0, label_smoothing=0.1)


@pytest.mark.parametrize("V", [3000, 9000])  # one workgroup, rows cut into pieces
def test_preference_pairs_and_rows_left_out(V):
    """A pair of weight 0 whose rows are NaN, rows outside every sequence that
    are NaN: the rest as if they were not there, their gradient 0."""
    torch = torch_mod()
    rng = np.random.default_rng(4)
    Y, _ = _make_Y(rng, 14, V, torch.bfloat16)
    labels = rng.integers(0, V, 14)
    off = [2, 4, 6, 9, 12]
    clean = _run_preference(Y, labels, off, pair_weight=[1.0, 0.0])
    Y[6:] = float("nan")
    Y[:2] = float("inf")
    labels = labels.copy()
    labels[[0, 1, 12, 13]] = -100
    got = _run_preference(Y, labels, off, pair_weight=[1.0, 0.0])
    assert got["loss"] == clean["loss"] and np.array_equal(got["dY"], clean["dY"])
    assert not got["dY"][6:].any() and not got["dY"][:2].any() and got["dY"][2:6].any()
    assert not got["logp"][[0, 1, 12, 13]].any() and np.isnan(got["chosen_reward"][1])


@pytest.mark.parametrize("V", [400, 12000])  # one workgroup, rows cut into pieces
def test_preference_offsets_outside_the_rows_end_at_their_borders(V):
    torch = torch_mod()
    rng = np.random.default_rng(12)
    Y, Y64 = _make_Y(rng, 6, V, torch.float32)
    labels = rng.integers(0, V, 6)
    for off in ([-5, 3, 9], [0, 2, 100], [-7, -3, 4, 2 ** 31 - 1, 2 ** 31 - 1], [-(2 ** 31), 6, 6]):
        got = _run_preference(Y, labels, off)
        _check_preference(got, Y64, labels, np.array(off, np.int64), False)
    # descending: the sequence is empty, the others have the rows that are theirs
    got = _run_preference(Y, labels, [4, 2, 6])
    assert got["chosen_reward"][0] == 0 and np.isfinite(got["dY"]).all()


# ------------------------------------------------------- streams and graphs ---

def test_losses_on_another_stream_and_in_a_graph():
    """The stream argument (a torch stream, a raw handle), and a captured graph
    of both losses replayed on changed inputs, in turn with eager calls."""
    torch = torch_mod()
    ah = ah_mod()
    rng = np.random.default_rng(13)
    N, V = 24, 30011
    Y, _ = _make_Y(rng, N, V, torch.bfloat16)
    labels, A = _dev(rng.integers(0, V, N), torch.int32), _dev(rng.normal(0, 1, N), torch.float32)
    off = _dev([0, 9, 12, 20, 24], torch.int32)

    def both(**kw):
        p = ah.archead_policy_loss(Y, labels, A, **kw)
        q = ah.archead_preference_loss(Y, labels, off, **kw)
        return [p[k] for k in sorted(p)] + [q[k] for k in sorted(q)]

    want = [t.clone() for t in both()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = both(stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs: their workspaces are their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs))
    for i in range(4):
        Y.copy_(torch.as_tensor(rng.normal(0, 3, (N, V)).astype(np.float32)))
        want = [t.clone() for t in both()]
        for g, outs in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_binding_refusals():
    torch = torch_mod()
    ah = ah_mod()
    Y = torch.zeros((4, 10), device="cuda")
    labels, A = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    bad = [lambda: ah.archead_policy_loss(Y.cpu(), labels, A), lambda: ah.archead_policy_loss(Y.t(), labels, A),
           lambda: ah.archead_policy_loss(Y, labels.long(), A), lambda: ah.archead_policy_loss(Y, labels, A[:3]),
           lambda: ah.archead_policy_loss(Y, labels, A.double()), lambda: ah.archead_policy_loss(Y, labels, A.cpu()),
           lambda: ah.archead_policy_loss(Y, labels, A, dY=Y.bfloat16(), dY_dtype=torch.float32),
           lambda: ah.archead_preference_loss(Y, labels, off[:2]),
           lambda: ah.archead_preference_loss(Y, labels, off, pair_weight=A),
           lambda: ah.archead_policy_loss(Y, labels, A, workspace=torch.zeros(4, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    for f, status in [(lambda: ah.archead_policy_loss(Y.half(), labels, A), 4),
                      (lambda: ah.archead_policy_loss(Y, labels, A, kl_coef=0.1), 1),
                      (lambda: ah.archead_policy_loss(Y, labels, A, dY=Y[:, :9]), 5),
                      (lambda: ah.archead_policy_loss(Y, labels, A, inv_temperature=0.0), 9),
                      (lambda: ah.archead_preference_loss(Y, labels, off, label_smoothing=0.6), 9),
                      (lambda: ah.archead_policy_loss(torch.zeros((4, 20000), device="cuda"), labels, A,
                                                      workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 7)]:
        with pytest.raises(ah.ArcheadError) as e:
            f()
        assert e.value.status == status
