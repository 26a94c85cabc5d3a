"""The losses' vectors must not share bytes with an output (no GPU: refused before the first HIP call)."""
import ctypes

import pytest

from tests.test_abi import ah  # noqa: F401
from tests.test_abi_loss import FAKE, N, V, _Call


def _vectors(call):
    """name -> (struct, field, elements) of every vector of the call"""
    pairs = 2
    inputs = dict(labels=N, ref_logp=N, weight=N)
    outputs = dict(loss=1, logp=N)
    if call.pairs:
        inputs.update(offsets=2 * pairs + 1, pair_weight=pairs)
        outputs.update(chosen_reward=pairs, rejected_reward=pairs)
    else:
        inputs.update(advantage=N, old_logp=N)
        outputs.update(row_loss=N)
    return inputs, outputs


@pytest.mark.parametrize("pairs", [False, True])
def test_outputs_that_share_bytes_are_refused(ah, pairs):  # noqa: F811
    inputs, outputs = _vectors(_Call(ah, pairs))
    for out, n_out in outputs.items():
        for other, n in {**inputs, **outputs}.items():
            if other == out:
                continue
            for elements, status in ((0, 5), (n - 1, 5), (n, 7), (-n_out, 7), (1 - n_out, 5)):
                call = _Call(ah, pairs)
                at = getattr(call.inp if other in inputs else call.out, other)
                setattr(call.out, out, at + 4 * elements)
                call.ws_bytes = 0  # what is not refused for its vectors ends at the workspace
                assert call() == status, (out, other, elements)


@pytest.mark.parametrize("pairs", [False, True])
def test_vectors_in_the_workspace_or_the_gradient_are_refused(ah, pairs):  # noqa: F811
    inputs, outputs = _vectors(_Call(ah, pairs))
    for name in (*inputs, *outputs):
        for at, status in (("ws", 5), ("dY", 5)):
            call = _Call(ah, pairs)
            where = call.ws if at == "ws" else call.dY.data + 4 * (N * V - 1)
            setattr(call.inp if name in inputs else call.out, name, where)
            assert call() == status, (name, at)
    call = _Call(ah, pairs)  # an output in the logits, which a later kernel may read
    call.out.logp = FAKE
    assert call() == 5
