"""h of rows whose product of sum and weight leaves fp32 though h does not.

h = s inv w has the roundings of the factor inv and of two products, 2^-24 each,
and the one to bf16, 2^-8: 2^-8 + 2^-22 of it allowed, and 2^-134 (half a step
where bf16 is subnormal, and an fp32 product there) on top.
"""
import numpy as np
import pytest

from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("D", [96, 300, 1001, 4096, 20000])
def test_h_where_sum_times_weight_leaves_the_range(D, residual):
    log(f"norm products D={D} residual={residual}")
    torch, ah = torch_mod(), ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(D)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    # (row, weight): products above 2^128 and below 2^-126, h between
    for row, weight, eps in ((83, 50, 1e-6), (125, 60, 1e-6), (100, 30, 1e-6), (120, -60, 1e-6), (0, 0, 1e-6), (-60, -80, 1e-36),
                             (-100, -30, 1e-44), (-125, 40, 1e-6), (60, -125, 1e-6)):
        x = (randn(5, D).clamp(-3.9, 3.9) * 2.0 ** row).bfloat16()
        r = (randn(5, D).clamp(-3.9, 3.9) * 2.0 ** row * 0.5).bfloat16() if residual else None
        w = (randn(D) * 2.0 ** weight).bfloat16()
        x[3] = 0
        got = ah.archead_rmsnorm(x, weight=w, residual=r, eps=eps, outputs=("h", "inv_rms", "sum"))
        s = got["sum"].double().cpu().numpy() if residual else x.double().cpu().numpy()
        assert np.isfinite(s).all()
        inv = 1.0 / np.sqrt(np.mean(s * s, 1, keepdims=True) + float(np.float32(eps)))
        want = s * inv * w.double().cpu().numpy()
        err = np.abs(got["h"].double().cpu().numpy() - want)
        tol = (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -134
        assert np.abs(want).max() < 2.0 ** 127
        assert (err <= tol).all(), (row, weight, float(np.nanmax(err / tol)))


def test_h_of_ordinary_rows_is_the_same_product():
    """Rows whose products stay in range: h equals bf16(fp32(fp32(s w) inv))."""
    torch, ah = torch_mod(), ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn((300, 1001), generator=gen, device="cuda") * 3).bfloat16()
    w = torch.randn(1001, generator=gen, device="cuda").bfloat16()
    got = ah.archead_rmsnorm(x, weight=w, outputs=("h", "inv_rms"))
    assert torch.equal(got["h"], (x.float() * w.float() * got["inv_rms"][:, None]).bfloat16())


def test_rows_that_are_not_finite_keep_the_formula():
    """inv is 0 beside an infinity: what is finite in such a row gives 0 and
    the infinity NaN; a NaN makes the row NaN."""
    torch, ah = torch_mod(), ah_mod()
    x = torch.full((3, 200), 2.0 ** 100, device="cuda").bfloat16()
    x[0, 5], x[1, 7] = float("inf"), float("nan")
    w = torch.full((200,), 2.0 ** 60, device="cuda").bfloat16()
    h = ah.archead_rmsnorm(x, weight=w)["h"]
    assert torch.isnan(h[0, 5]) and not h[0, :5].any() and not h[0, 6:].any()
    assert torch.isnan(h[1]).all()
    assert (h[2] == 2.0 ** 60).all()


@pytest.mark.parametrize("D", [96, 1001, 20000])
def test_rows_that_are_read_again_in_place(D):
    """Sum and h in the place of x or the residual, and no sum kept at all."""
    import ctypes
    torch, ah = torch_mod(), ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(D)
    N = 9
    scale = 2.0 ** torch.tensor([0.0, 83, 100, 125, 0, 83, -100, 110, 60], dtype=torch.float64, device="cuda")[:, None]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64).clamp(-3.9, 3.9)  # noqa: E731
    x, r = (randn(N, D) * scale).bfloat16(), (randn(N, D) * scale * 0.5).bfloat16()
    w = (randn(D) * 2.0 ** 50).bfloat16()
    want = ah.archead_rmsnorm(x, weight=w, residual=r, outputs=("h", "codes"))
    s = want["sum"]
    assert torch.isfinite(want["h"]).all() and torch.isnan(want["scale"][3])
    plain = ah.archead_rmsnorm(s, weight=w, outputs=("h",))["h"]
    assert torch.equal(plain, want["h"])
    y = s.clone()
    assert torch.equal(ah.archead_rmsnorm(y, weight=w, h=y)["h"], plain)
    for sum_at, h_at in (("x", "r"), ("r", "x"), ("x", None), ("r", None), (None, "x"), (None, "r")):
        t = {"x": x.clone(), "r": r.clone(), None: None}
        got = ah.archead_rmsnorm(t["x"], weight=w, residual=t["r"], outputs=("h", "codes"), sum=t[sum_at], h=t[h_at])
        for k in ("sum", "h", "codes"):
            assert torch.equal(got[k], want[k]), (sum_at, h_at, k)
    for h_at in ("x", "r", "new"):  # the C call keeps the sum only where it is asked to
        t = {"x": x.clone(), "r": r.clone(), "new": torch.full_like(x, 7.0)}
        X, R, H = (ah._tensor(v) for v in (t["x"], t["r"], t[h_at]))
        inp = ah.ArcheadRmsnormInputs(ctypes.addressof(X), ctypes.addressof(R), w.data_ptr(), 1e-6)
        out = ah.ArcheadRmsnormOutputs(None, ctypes.addressof(H), None, None, None)
        assert ah.lib.archead_rmsnorm(inp, out, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(t[h_at], want["h"]), h_at
