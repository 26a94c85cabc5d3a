"""CPU oracle of the norm in front of the head, the INT8 product and the cross
entropy through a packed head -- TEST INFRASTRUCTURE ONLY.

In fp64 from their definitions (the same ones ``include/archead.h`` states).
Pinned by ``tests/test_front_oracle.py`` against differences, closed forms and
whole-number arithmetic.
"""
from __future__ import annotations

import numpy as np

from .archead_oracle import w_hat, w_hat_alt


def round_bf16(x):
    """fp32 rounding, then bf16 rounding (half to even), as fp64."""
    with np.errstate(over="ignore"):
        b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    up = ((b >> 16) & 1) + 0x7FFF
    r = np.where((b & 0x7FFFFFFF) > 0x7F800000, b | 0x400000, b + up) & np.uint32(0xFFFF0000)
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


def rmsnorm(x, residual=None, weight=None, eps=1e-6):
    """dict sum, h, codes (int64), scale, inv_rms (fp64) of bf16 values in fp64."""
    s = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if residual is not None:
            s = round_bf16(s + np.asarray(residual, np.float64))
        w = np.ones(s.shape[1]) if weight is None else np.asarray(weight, np.float64)
        inv = 1.0 / np.sqrt(np.mean(s * s, 1) + eps)
        t = s * w
        t = np.where(np.isinf(t.astype(np.float32)), np.inf * t, t)  # products are fp32
        m = np.abs(t).max(1)
        fine = np.isfinite(t).all(1) & np.isfinite(s).all(1)
        q = 127.0 * t / np.where(m > 0, m, 1.0)[:, None]
        codes = np.where(fine[:, None], np.rint(np.where(fine[:, None], q, 0.0)), 0.0).astype(np.int64)
        scale = np.where(fine, m * inv / 127.0, np.nan)
        return dict(sum=s, h=t * inv[:, None], codes=codes, scale=scale, inv_rms=inv)


def rmsnorm_backward(dh, s, inv_rms, weight=None, dsum=None):
    """dict dx, dweight (fp64)."""
    dh, s, inv = np.asarray(dh, np.float64), np.asarray(s, np.float64), np.asarray(inv_rms, np.float64)[:, None]
    w = np.ones(s.shape[1]) if weight is None else np.asarray(weight, np.float64)
    g = dh * w
    dx = inv * (g - s * inv ** 2 * np.mean(g * s, 1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dict(dx=dx, dweight=(dh * s * inv).sum(0))


def logits_int8(codes, scale, head):
    """diag(scale) codes W_hat^T of a row-INT8 head."""
    return (np.asarray(codes, np.float64) @ w_hat_alt(head).T) * np.asarray(scale, np.float64)[:, None]


def cross_entropy(H, labels, head, weight=None, inv_temperature=1.0, W=None):
    """dict loss, logp, dH (fp64); H: fp64 values, W: w_hat(head) if it is at hand."""
    H, labels = np.asarray(H, np.float64), np.asarray(labels, np.int64)
    N, V = len(H), head.V
    W = w_hat(head) if W is None else W
    w = np.ones(N) if weight is None else np.asarray(weight, np.float64)
    on = w != 0
    logp, dH = np.zeros(N), np.zeros(H.shape)
    for n in np.flatnonzero(on):
        with np.errstate(all="ignore"):
            z = (W @ H[n]) * inv_temperature
            l = labels[n]
            if not (0 <= l < V) or not np.isfinite(z).all():
                logp[n], dH[n] = np.nan, np.nan
                continue
            rest = np.delete(z, l)
            top = rest.max() if V > 1 else -np.inf
            S = np.exp(rest - top).sum() if V > 1 else 0.0
            # 1 - p of the label and log p, each without the other's cancellation
            d = top + np.log(S) - z[l] if V > 1 else -np.inf
            logp[n] = -np.logaddexp(0.0, d)
            q = np.exp(-np.logaddexp(0.0, -d)) if V > 1 else 0.0
            p = np.insert(np.exp(rest - top) / S * q if V > 1 else rest, l, -q)
            dH[n] = w[n] * inv_temperature * (p @ W)
    return dict(loss=-np.sum(np.where(on, w * logp, 0.0)), logp=logp, dH=dH)
