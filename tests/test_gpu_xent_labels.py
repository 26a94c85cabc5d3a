"""Labels at the ends of int32 in rows that count: NaN there, and every other
row as without them."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import ah_mod, torch_mod
from tests.test_gpu_xent import _head, _hidden

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [5, 32, 40, 200])
def test_labels_at_the_ends_of_their_type(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 1000, 256
    h, head = _head(3, V, D, 16, 8, 64)
    labels = np.random.default_rng(N).integers(0, V, N)
    H = _hidden(4, N, D, oracle.w_hat(h), labels)
    good = torch.from_numpy(labels).int().cuda()
    want = ah.archead_cross_entropy(H, good, head)
    bad = good.clone()
    wrong = [-2 ** 31, 2 ** 31 - 1, -2 ** 31 + 500, 2 ** 24, -V][:N]
    bad[:len(wrong)] = torch.tensor(wrong, dtype=torch.int32, device="cuda")
    got = ah.archead_cross_entropy(H, bad, head)
    k = len(wrong)
    assert torch.isnan(got["loss"]) and torch.isnan(got["logp"][:k]).all() and torch.isnan(got["dH"][:k]).all()
    assert torch.equal(got["logp"][k:], want["logp"][k:]) and torch.equal(got["dH"][k:], want["dH"][k:])
