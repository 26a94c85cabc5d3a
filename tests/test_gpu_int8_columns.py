"""Every column of the head through archead_logits_int8, one at a time: the
order in which codes and hidden states meet, for each way through the kernels."""
import numpy as np
import pytest

import synth
from tests.gpu_helpers import ah_mod, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 3, 8, 9, 64, 100, 300])
@pytest.mark.parametrize("D", [128, 512, 640])
def test_unit_rows_give_every_column(N, D):
    torch, ah = torch_mod(), ah_mod()
    V = 100
    h = synth.draw_alt_head(np.random.default_rng(N), 2, V, D, 64)
    h.scales[:] = 1.0
    head = ah.PackedHead.from_components(h)
    want = torch.from_numpy(h.codes.astype(np.float32)).cuda()
    one = torch.ones(N, device="cuda")
    for k0 in range(0, D, N):
        k = torch.arange(k0, k0 + N, device="cuda") % D
        X = torch.zeros((N, D), dtype=torch.int8, device="cuda")
        X[torch.arange(N, device="cuda"), k] = 1
        assert torch.equal(ah.archead_logits_int8(X, one, head), want[:, k].T), k0
