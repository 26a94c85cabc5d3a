"""Scales of hidden states at the ends of fp32's range in archead_logits_int8.

A logit is (sum s[v]) scale[n]: the sum rounded where it is above 2^24, its
product with the row's fp16 scale (between 2^-24 and 2^46 or 0, never out of
range) and the one with the token's, 2^-24 each: 2^-22 of the logit, 2^-8 more
for bf16, and half a step of a subnormal result.
"""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N", [3, 8, 45, 100, 150, 300])
def test_scales_of_any_size(N, dtype):
    log(f"int8 scales N={N} {dtype}")
    torch, ah = torch_mod(), ah_mod()
    V, D = 517, 384
    rng = np.random.default_rng(N)
    h = synth.draw_alt_head(rng, 2, V, D, 64)
    h.scales[:] = np.resize(np.array([1e-5, 6e-8, 1e-3, 1.0, 10.0, 60000.0], np.float16), V)
    head = ah.PackedHead.from_components(h)
    X = rng.integers(-128, 128, (N, D), dtype=np.int8)
    X[:, 7:] *= rng.random((N, 1)) < 0.5  # rows of small sums
    X[2] = 0
    s = np.resize(np.array([6e-36, 1e38, 1e38, 2e-38, 1e-42, 3e38, 1.0, 1e-30, 1e30, 0.0]), N).astype(np.float32)
    Y = torch.full((N, V), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    ah.archead_logits_int8(torch.from_numpy(X).cuda(), torch.from_numpy(s).cuda(), head, Y)
    want, got = oracle.logits_int8(X, s.astype(np.float64), h), Y.double().cpu().numpy()
    bf16 = dtype == "bfloat16"
    rel = 2.0 ** -22 + (2.0 ** -8 if bf16 else 0)
    most = 2.0 ** 128 * (1 - rel)
    inside, outside = np.abs(want) < most, np.abs(want) > 2.0 ** 128
    assert inside.sum() > want.size // 2 and (N < 6 or outside.any())
    tol = rel * np.abs(want) + (2.0 ** -134 if bf16 else 2.0 ** -149)
    bad = ~(np.abs(got - want) <= tol) & inside
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    assert np.isinf(got[outside]).all() and (np.sign(got[outside]) == np.sign(want[outside])).all()
    assert not got[2].any()  # 0 times a finite scale
