"""The norm's gradient of rows at the ends of bf16's range, which the forward
pass takes: factors and sums as they are for ordinary rows.

Tolerances as in test_gpu_norm.py: at most 16 fp32 roundings, 2^-24 each, of
terms of the size of inv |g|, inv |s| inv sum_d|g s inv| / D and |dsum| for dx
(2^-20), one for each row that a thread adds (N here) and four more for dweight,
and bf16's own 2^-8 (2^-134 where it is subnormal).  s inv is a number of
ordinary size, and rounding it is one of the 16.
"""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("through", [True, False])
@pytest.mark.parametrize("D", [96, 129, 1001, 2048, 4096, 12001, 32768])
def test_gradient_of_rows_at_the_ends_of_the_range(D, through):
    log(f"norm backward of extreme rows D={D} through={through}")
    torch, ah = torch_mod(), ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(D)
    scale = 2.0 ** torch.tensor([90.0, 120.0, 125.0, 63.0, 0.0, -63.0, -100.0, -125.0], dtype=torch.float64, device="cuda")
    N = len(scale)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    x = (randn(N, D).clamp(-3.9, 3.9) * scale[:, None]).bfloat16()
    x[2, 0] = 3.38e38
    w = randn(D).bfloat16()
    # gradients of which dx is of ordinary size where the row is large
    dh = (randn(N, D) * 8.0 * scale.clamp(min=1.0)[:, None] ** 0.5).bfloat16()
    ds = randn(N, D).bfloat16() if through else None
    inv = ah.archead_rmsnorm(x, weight=w, outputs=("inv_rms",))["inv_rms"]
    assert torch.isfinite(x).all() and torch.isfinite(dh).all() and torch.isfinite(inv).all() and (inv > 0).all()
    got = ah.archead_rmsnorm_backward(dh, x, inv, weight=w, dsum=ds)
    g64, s64, i64 = _np(dh), _np(x), _np(inv)[:, None]
    want = oracle.rmsnorm_backward(g64, s64, i64[:, 0], _np(w), None if ds is None else _np(ds))
    g, unit = np.abs(g64 * _np(w)), np.abs(s64 * i64)
    size = i64 * (g + unit * (g * unit).mean(1, keepdims=True)) + (0 if ds is None else np.abs(_np(ds)))
    tol = 2.0 ** -20 * size
    tol = tol + 2.0 ** -8 * (np.abs(want["dx"]) + tol) + 2.0 ** -134
    err = np.abs(_np(got["dx"]) - want["dx"])
    assert (err <= tol).all(), [float((err / tol)[n].max()) for n in range(N)]
    terms = np.abs(g64 * s64 * i64).sum(0)
    tol = (N + 4) * 2.0 ** -24 * terms + 2.0 ** -24 * np.abs(want["dweight"]) + 2.0 ** -149
    assert (np.abs(_np(got["dweight"]) - want["dweight"]) <= tol).all()
