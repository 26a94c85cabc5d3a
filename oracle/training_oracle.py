"""CPU oracle of training through a frozen packed head -- TEST INFRASTRUCTURE ONLY.

The clipped policy loss with a KL term, the preference loss over pairs of
sequences (both with their gradient on the logits) and the gradient of the
hidden states, dH = dY W_hat, in fp64 from their definitions (the same ones
``include/archead.h`` states).  Pinned by ``tests/test_training_oracle.py``
against differences, closed forms and brute force.
"""
from __future__ import annotations

import numpy as np

from .archead_oracle import w_hat

PREF_SIGMOID, PREF_SQUARED = 0, 1


def _log_softmax(Y, labels, inv_temperature):
    """(log softmax [N, V], label log-probabilities); NaN rows where a label is
    outside [0, V) or the row has NaN, +inf or nothing above -inf."""
    z = np.asarray(Y, np.float64) * inv_temperature
    V = z.shape[1]
    labels = np.asarray(labels, np.int64)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = z.max(1, keepdims=True)
        q = z - top
        q = q - np.log(np.exp(q).sum(1, keepdims=True))
    bad = (labels < 0) | (labels >= V)
    lp = q[np.arange(len(z)), np.where(bad, 0, labels)]
    lp = np.where(bad, np.nan, lp)
    q[np.isnan(lp)] = np.nan
    return q, lp


def _gradient(Y, labels, q, lp, slope, inv_temperature):
    """slope_n s (one-hot - softmax); zero rows where the slope is zero."""
    dY = np.zeros(q.shape)
    for n in np.flatnonzero(slope != 0):
        if np.isnan(slope[n]):
            dY[n] = np.nan
            continue
        dY[n] = -np.exp(q[n]) * slope[n] * inv_temperature
        dY[n, labels[n]] = -np.expm1(lp[n]) * slope[n] * inv_temperature
    return dY


def policy_loss(Y, labels, advantage, old_logp=None, ref_logp=None, weight=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, inv_temperature=1.0):
    """dict loss, logp, row_loss, dY (fp64)."""
    N = len(Y)
    w = np.ones(N) if weight is None else np.asarray(weight, np.float64)
    on = w != 0
    Yc = np.where(on[:, None], np.asarray(Y, np.float64), 0.0)
    q, lp = _log_softmax(Yc, np.where(on, labels, 0), inv_temperature)
    A = np.asarray(advantage, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.where(np.isnan(lp), lp, 1.0) if old_logp is None else np.exp(lp - np.asarray(old_logp, np.float64))
        kept = np.minimum(np.maximum(r, 1.0 - clip_low), 1.0 + clip_high)
        plain = ~(kept * A < r * A)
        row = -np.where(plain, r * A, kept * A)
        slope = -np.where(plain, r * A, 0.0)
        if kl_coef:
            d = np.asarray(ref_logp, np.float64) - lp
            row = row + kl_coef * (np.expm1(d) - d)
            slope = slope - kl_coef * np.expm1(d)
    row, lp, slope = np.where(on, row, 0.0), np.where(on, lp, 0.0), np.where(on, w * slope, 0.0)
    return dict(loss=np.sum(np.where(on, w * row, 0.0)), logp=lp, row_loss=row,
                dY=_gradient(Y, labels, q, lp, slope, inv_temperature))


def preference_loss(Y, labels, offsets, ref_logp=None, weight=None, pair_weight=None, beta=0.1, label_smoothing=0.0,
                    inv_temperature=1.0, kind=PREF_SIGMOID):
    """dict loss, logp, chosen_reward, rejected_reward, dY (fp64)."""
    N, B = len(Y), (len(offsets) - 1) // 2
    off = np.clip(np.asarray(offsets, np.int64), 0, N)
    w = np.ones(N) if weight is None else np.asarray(weight, np.float64)
    on = (w != 0) & (np.arange(N) >= off[0]) & (np.arange(N) < off[2 * B])
    Yc = np.where(on[:, None], np.asarray(Y, np.float64), 0.0)
    q, lp = _log_softmax(Yc, np.where(on, labels, 0), inv_temperature)
    lp = np.where(on, lp, 0.0)
    ref = np.zeros(N) if ref_logp is None else np.asarray(ref_logp, np.float64)
    terms = np.where(on, np.where(on, w, 0.0) * (lp - ref), 0.0)
    S = np.array([terms[off[i]:off[i + 1]].sum() for i in range(2 * B)])
    h = S[0::2] - S[1::2]
    if kind == PREF_SIGMOID:
        loss = (1 - label_smoothing) * np.logaddexp(0, -beta * h) + label_smoothing * np.logaddexp(0, beta * h)
        slope = beta * (label_smoothing - np.exp(-np.logaddexp(0, beta * h)))
    else:
        loss, slope = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
    if pair_weight is not None:
        pw = np.asarray(pair_weight, np.float64)
        loss, slope = np.where(pw != 0, pw * loss, 0.0), np.where(pw != 0, pw * slope, 0.0)
    coef = np.zeros(N)
    for i in range(B):
        coef[off[2 * i]:off[2 * i + 1]] = slope[i]
        coef[off[2 * i + 1]:off[2 * i + 2]] = -slope[i]
    coef = np.where(on, coef * np.where(on, w, 0.0), 0.0)
    return dict(loss=loss.sum(), logp=lp, chosen_reward=beta * S[0::2], rejected_reward=beta * S[1::2],
                dY=_gradient(Y, labels, q, lp, coef, inv_temperature))


def logits_backward(dY, head, v_chunk=8192):
    """dH = dY W_hat in fp64."""
    dY = np.asarray(dY, np.float64)
    out = np.zeros((dY.shape[0], head.D))
    for v0 in range(0, head.V, v_chunk):
        v1 = min(head.V, v0 + v_chunk)
        out += dY[:, v0:v1] @ w_hat(head, v0, v1)
    return out
