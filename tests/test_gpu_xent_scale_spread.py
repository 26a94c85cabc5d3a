"""Cross entropy of more than 32 rows through heads whose row scales lie far
apart.

The product takes s_R times a power of two in fp16, one for the head, which
brings 2040 times the largest to [2^14, 2^15): what is below 2^-14 then has a half
step of 2^-25, which is 2^-28 of the largest s_R at most; and s_Ac, s_Aw likewise,
the largest to [1/2, 1), a half step being 2^-24 of the largest at most.  (With the
largest s_R below 16, s_A below 1, the power is 1 or more and nothing is lost.)
Their products with the codes and operands are rounded to fp16, 2^-11, or by
2^-25 where subnormal: of q4 c8 s_R that is 2^-39 of 2040 times the largest s_R,
and of e s_A, where a row's largest e is at least 2^10, 2^-34 of the largest s_A for
every entry.  So dH may be off, beside the bounds of test_gpu_xent.py, by |w| tau
times
    sum_v p_v (|q4 c8| 2^-28 max s_R + |A| |B| 2^-24 max s_A)  [where the power is below 1]
    + q (2040 2^-39 max s_R + 2^-34 / S sum_v |A| |B| max s_A).
"""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("N", [40, 200])
def test_row_scales_far_apart(N, large):
    log(f"xent scales N={N} large={large}")
    torch, ah = torch_mod(), ah_mod()
    V, D, g, r = 1500, 256, 64, 16
    rng = np.random.default_rng(N)
    h = synth.draw_head(rng, V, D, r // 2, r // 2, g)
    # s_R and s_A from 2^-20 (2^-13) of the largest to it; hidden states small enough for logits of a few
    top_R, top_A = (40000.0, 500.0) if large else (0.05, 0.4)
    h.s_R[...] = (top_R * 2.0 ** -rng.uniform(0, 20, V)).astype(np.float16)
    for s in (h.s_Ac, h.s_Aw):
        s[...] = (top_A * 2.0 ** -rng.uniform(0, 13, V)).astype(np.float16)
    h.s_R[:2], h.s_Ac[:2], h.s_Aw[:2] = np.float16(top_R), np.float16(top_A), np.float16(top_A)
    head = ah.PackedHead.from_components(h)
    W = oracle.w_hat(h)
    H = rng.normal(0, 1, (N, D))
    H *= (rng.choice([0.5, 2.0, 6.0], N) / np.abs(H @ W.T).max(1))[:, None]
    X = torch.from_numpy(H.astype(np.float32)).cuda().bfloat16()
    H = X.double().cpu().numpy()
    labels = rng.integers(0, V, N)
    got = ah.archead_cross_entropy(X, torch.from_numpy(labels).int().cuda(), head)
    want = oracle.cross_entropy(H, labels, h, W=W)
    q = -np.expm1(want["logp"])
    codes = np.abs(h.q4.astype(np.float64)) * np.repeat(h.c8.astype(np.float64), g, 1)
    low = np.zeros_like(codes)  # |A| |B| without s_A
    Wabs = codes * h.s_R.astype(np.float64)[:, None]
    for A, s_A, B, s_B in ((h.A_c, h.s_Ac, h.B_c, h.s_Bc), (h.A_w, h.s_Aw, h.B_w, h.s_Bw)):
        part = np.abs(A.astype(np.float64)) @ (np.abs(B.astype(np.float64)) * np.repeat(np.abs(s_B.astype(np.float64)), g, 1))
        low += part
        Wabs += part * s_A.astype(np.float64)[:, None]
    eps = (D / 16 + r / 16 + 32) * 2.0 ** -24 * (np.abs(H) @ Wabs.T).max(1)
    err = np.abs(got["logp"].double().cpu().numpy() - want["logp"])
    assert (err <= q * (2 * eps + 2.0 ** -18) + 2.0 ** -24 * np.abs(want["logp"])).all()
    z = H @ W.T
    z[np.arange(N), labels] = -np.inf
    e = np.exp(z - z.max(1, keepdims=True))
    S = e.sum(1, keepdims=True)
    p = q[:, None] * e / S
    T = p @ Wabs + q[:, None] * Wabs[labels]
    rel = 2.0 ** -10 + 4 * eps[:, None] + 2.0 ** -17 + (V / 16 + 128) * 2.0 ** -24 + r * 2.0 ** -23 + 3 * 2.0 ** -18
    most_R, most_A = float(h.s_R.max()), float(max(h.s_Ac.max(), h.s_Aw.max()))
    tol = rel * T + 2.0 ** -34 * q[:, None] / S * (Wabs.sum(0) + most_A * low.sum(0))
    tol = tol + q[:, None] * 2040 * 2.0 ** -39 * most_R
    if most_R >= 16:
        tol = tol + p @ codes * 2.0 ** -28 * most_R
    if most_A >= 1:
        tol = tol + p @ low * 2.0 ** -24 * most_A
    tol = tol + 2.0 ** -8 * (np.abs(want["dH"]) + tol) + 2.0 ** -134
    err = np.abs(got["dH"].double().cpu().numpy() - want["dH"])
    assert (err <= tol).all(), float((err / tol).max())
    log(f"  dH error / bound {(err / tol).max():.3f}")
