"""The losses' and the backward's stream argument: one of another device is refused (no GPU:
the call ends before its first argument is looked at more closely)."""
import types

import pytest

from tests.test_abi import ah  # noqa: F401


@pytest.mark.parametrize("name", ["archead_policy_loss", "archead_preference_loss", "archead_logits_backward"])
def test_a_stream_of_another_device_is_refused(ah, name):  # noqa: F811
    torch = pytest.importorskip("torch")
    first = types.SimpleNamespace(device=torch.device("cuda", 0))
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        getattr(ah, name)(first, None, None, stream=stream)
