"""Cross entropy of more than 32 rows over several pieces of the vocabulary:
the running exponent, operands that are moved to it, and sums that are brought
along, for 2, 4, 6 and 8 row tiles a workgroup as the rows that count choose
them, for every group size, and in a second pass of rows.

A piece is 2^28 bytes of operands: 256 entries of the vocabulary are 2^17 of them
for 256 rows.  Half of the rows have logits that rise along the vocabulary, so
that exponents move from one piece to the next.  Bounds: those of
test_gpu_xent.py, for 60 of the rows that count.
"""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import ah_mod, log, torch_mod
from tests.test_gpu_xent import _check, _head

pytestmark = pytest.mark.gpu


def _hidden(rng, W, N, D, labels, V):
    H = rng.normal(0, 1, (N, D))
    late = rng.integers(V // 2, V, N)
    rise = rng.choice([0.0, 0.0, 6.0, 25.0, 80.0], N)
    H += (rise / (W[late] ** 2).sum(1))[:, None] * W[late]
    return H, np.where(rng.random(N) < 0.3, late, labels)


def _run(V, D, r_c, r_r, g, N, count, look=60):
    log(f"xent pieces V={V} D={D} r_c={r_c} r_r={r_r} g={g} N={N} count={count}")
    torch, ah = torch_mod(), ah_mod()
    h, head = _head(V + N, V, D, r_c, r_r, g)
    W = oracle.w_hat(h)
    rng = np.random.default_rng(count)
    H, labels = _hidden(rng, W, N, D, rng.integers(0, V, N), V)
    del W
    on = np.zeros(N, bool)
    on[rng.permutation(N)[:count]] = True
    weight = np.where(on, rng.uniform(0.5, 1.5, N), 0.0)
    X = torch.from_numpy(np.where(on[:, None], H, np.nan).astype(np.float32)).cuda().bfloat16()
    lab = torch.from_numpy(np.where(on, labels, -100)).int().cuda()
    w = torch.from_numpy(weight.astype(np.float32)).cuda()
    need = ah.archead_cross_entropy_workspace_bytes(V, D, r_c, r_r, g, N)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = ah.archead_cross_entropy(X, lab, head, weight=w, workspace=ws)
    off = torch.from_numpy(~on).cuda()
    assert not got["logp"][off].any() and not got["dH"][off].any()
    logp, w64 = got["logp"].double(), w.double()
    assert abs(got["loss"].item() + (w64 * logp).sum().item()) <= 2.0 ** -22 * (w64 * logp).abs().sum().item()
    rows = np.flatnonzero(on)
    if count > look:  # the last ones, which a second pass takes, and some of the others
        rows = np.unique(np.concatenate([rows[-look // 2:], rng.choice(rows, look // 2, replace=False)]))
    at = torch.from_numpy(rows).cuda()
    part = {"logp": got["logp"][at], "dH": got["dH"][at], "loss": -(w64 * logp)[at].sum()}
    _check(part, X[at], labels[rows], w[at], h, 1.0, f"V={V} count={count}")
    again = ah.archead_cross_entropy(X, lab, head, weight=w, workspace=ws)
    for k in got:
        assert torch.equal(again[k], got[k]), k


# V, D, r_c, r_r, g, N, rows that count: 2, 4 and 6 row tiles a workgroup; 8 of them, rows of a
# call decide; more rows that count than a pass takes
CASES = [
    (140001, 256, 16, 8, 32, 1000, 50), (140001, 256, 8, 40, 64, 1000, 115), (140001, 256, 0, 8, 128, 1000, 185),
    (140001, 256, 8, 0, 256, 1000, 250), (70001, 256, 8, 8, 32, 2000, 300), (33001, 128, 8, 8, 64, 4700, 4300),
]


@pytest.mark.parametrize("V,D,r_c,r_r,g,N,count", CASES)
def test_pieces(V, D, r_c, r_r, g, N, count):
    _run(V, D, r_c, r_r, g, N, count)
