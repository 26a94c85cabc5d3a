"""archead_logits_backward where rows are few or ranks many: on both sides of the vocabulary from
which the rows' maxima are a launch of their own, and the largest ranks with some tens of rows.
Tolerances as in test_gpu_backward.py."""
import numpy as np
import pytest

from tests.gpu_helpers import ah_mod, torch_mod
from tests.test_gpu_backward import _check, _gradient, _head

pytestmark = pytest.mark.gpu

# rows, and the longest vocabulary whose maxima the first kernel finds itself: eight rounds of
# eight columns of the lanes that a row has, 64 of them up to four rows, then by halves
OWN = [(1, 4096), (4, 4096), (5, 2048), (8, 2048), (9, 1024), (16, 1024), (17, 512), (32, 512)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("g", [32, 64, 128, 256])
@pytest.mark.parametrize("N,V", [(n, v + more) for n, v in OWN for more in (-5, 0, 1)])
def test_maxima_within_the_first_kernel_and_beside_it(N, V, g, dtype):
    torch = torch_mod()
    h, head = _head(V + g, V, 256, 16, 8, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N + V), N, V), device="cuda").to(getattr(torch, dtype))
    if N > 4:
        dY[2] = 0
    _check(head, h, dY, f"N={N} V={V} g={g} {dtype}")


@pytest.mark.parametrize("N,V", [(4, 4096), (4, 4097), (32, 512), (32, 513)])
def test_rows_that_are_not_finite_change_no_other(N, V):
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(V, V, 256, 8, 8, 64)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N), N, V), device="cuda").bfloat16()
    base = ah.archead_logits_backward(dY, head)
    dY[1, V - 1] = float("nan")
    dY[N - 2, 0] = float("inf")
    got = ah.archead_logits_backward(dY, head)
    torch.cuda.synchronize()
    keep = [i for i in range(N) if i not in (1, N - 2)]
    assert torch.equal(got[keep], base[keep]) and not torch.isfinite(got[[1, N - 2]].float()).any()


@pytest.mark.parametrize("N,V,D,r_c,r_r,g", [(40, 300, 256, 512, 512, 64), (33, 70, 384, 1024, 0, 32),
                                             (100, 130, 256, 0, 1024, 256), (257, 90, 512, 504, 520, 128)])
def test_largest_ranks_with_tens_of_rows(N, V, D, r_c, r_r, g):
    """r_c + r_r = 1024 in the last kernel that holds Z of its rows in LDS."""
    torch = torch_mod()
    h, head = _head(V, V, D, r_c, r_r, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N), N, V), device="cuda").bfloat16()
    _check(head, h, dY, f"N={N} r={r_c}+{r_r} g={g}")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [130, 1500])
@pytest.mark.parametrize("more", [1, 4, 17, 32])
def test_a_last_pass_of_few_rows(more, V, dtype):
    """Rows past 4096 are a pass of their own: as a call of those rows alone."""
    torch = torch_mod()
    ah = ah_mod()
    _, head = _head(V, V, 256, 8, 8, 64)
    gen = torch.Generator(device="cuda").manual_seed(more)
    dY = torch.randn((4096 + more, V), generator=gen, device="cuda").to(getattr(torch, dtype))
    got = ah.archead_logits_backward(dY, head)
    assert torch.equal(got[:4096], ah.archead_logits_backward(dY[:4096], head))
    assert torch.equal(got[4096:], ah.archead_logits_backward(dY[4096:], head))
    assert torch.isfinite(got.float()).all() and got[4096:].any(1).all()
