"""The policy loss of thousands of rows, several for each workgroup of its one launch, whose
columns past those held in registers are read again: against fp64 on the GPU, row by row.

Tolerances as in test_gpu_loss_digits.py (relative, of log p and of the gradient) but for log p of
rows without a likely label, which is a difference of numbers of its own size: absolute, as in
test_gpu_loss.py, u (|log p| + 2 spread + V / 256 + 3 * 74 + 4).
"""
import numpy as np
import pytest

from tests.gpu_helpers import ah_mod, torch_mod

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("y,dy,N,V", [("bfloat16", "bfloat16", 2100, 100003), ("bfloat16", "float32", 2053, 49999),
                                      ("float32", "bfloat16", 600, 60007)])
def test_policy_of_thousands_of_rows(y, dy, N, V):
    torch = torch_mod()
    ah = ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(N)
    s = 0.9
    Y = (torch.randn((N, V + 5), generator=gen, device="cuda") * 3).to(getattr(torch, y))[:, :V]
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    rows = torch.arange(N, device="cuda")
    labels[0], labels[1], labels[2] = V - 1, 98304, V // 8 * 8  # the last column, past those held, the rest
    labels = labels.clamp(max=V - 1)
    Y[rows, labels.long()] += (torch.rand(N, generator=gen, device="cuda") * 30).to(Y.dtype)
    Y[5, :9000] = -float("inf")
    Y[6, :9000] -= 60
    A = torch.randn(N, generator=gen, device="cuda")
    w = (torch.rand(N, generator=gen, device="cuda") < 0.8).float() / N
    got = ah.archead_policy_loss(Y, labels, A, weight=w, inv_temperature=s, dY_dtype=getattr(torch, dy))
    torch.cuda.synchronize()
    s, total = float(np.float32(s)), 0.0
    for a in range(0, N, 256):
        n = slice(a, min(N, a + 256))
        at = labels[n].long()[:, None]
        z = Y[n].double() * s
        top = z.max(1, keepdim=True)[0]
        own = (z.gather(1, at) - top)[:, 0]  # -inf where the label's column is masked
        E = torch.exp(own)
        e = torch.exp(z - top)
        e.scatter_(1, at, 0.0)
        S = e.sum(1)
        on = w[n] != 0
        logp = torch.where(on, torch.where(S < E, -torch.log1p(S / E), own - torch.log(S + E)), 0.0)
        finite = z.masked_fill(z == -float("inf"), float("inf"))
        spread = (z.max(1)[0] - finite.min(1)[0]) / np.log(2)
        rel = U * (3 * spread + 160)
        tol = torch.where(S < E, rel * logp.abs(), U * (logp.abs() + 2 * spread + V / 256 + 3 * 74 + 4))
        lp = got["logp"][n].double()
        assert ((lp == logp) | ((lp - logp).abs() <= tol)).all(), a
        coef = torch.where(on, A[n].double() * w[n].double(), 0.0) * s
        want = coef[:, None] * e / (S + E)[:, None]
        want.scatter_(1, at, (-coef * S / (S + E))[:, None])
        bound = (2 * rel + (2.0 ** -8 if dy == "bfloat16" else 0.0))[:, None] * want.abs() + 2.0 ** -126
        bad = (got["dY"][n].double() - want).abs() > bound
        assert not bad.any(), (a, bad.nonzero()[:4])
        assert not got["dY"][n][~on].any()
        want_loss = torch.where(on, -A[n].double(), 0.0)
        assert ((got["row_loss"][n].double() - want_loss).abs() <= U * want_loss.abs()).all()
        total += (w[n].double() * want_loss).sum().item()
    assert abs(got["loss"].item() - total) <= U * abs(total) + 1e-12
