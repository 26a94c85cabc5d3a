"""Argument checks and workspace sizes of the loss entry points (no GPU: every
call fails validation before the first HIP call)."""
import ctypes

import pytest

from tests.test_abi import ah  # noqa: F401

FAKE = 1 << 30  # an address that is never dereferenced
N, V = 4, 20000


def _up(x):
    return (x + 255) // 256 * 256


def _pieces(n, v):
    return max(1, min(64, -(-v // 2048), 12288 // n))


@pytest.mark.parametrize("n,v,b", [(4, 1024, 0), (1, 151936, 0), (4096, 151936, 0), (480, 151936, 4), (70000, 7, 3)])
def test_loss_workspace_bytes(ah, n, v, b):  # noqa: F811
    want = 0 if n <= 64 and n * v <= 65536 and b <= 64 else _up(n * _pieces(n, v) * 16) + _up(4 * n) + _up(16 * n) + _up(8 * n) + _up(4 * n + 4) + _up(8 * b)
    assert ah.archead_loss_workspace_bytes(n, v, b) == want


def test_loss_workspace_errors(ah):  # noqa: F811
    out = ctypes.c_uint64()
    f = ah.lib.archead_loss_workspace_bytes
    assert f(4, 10, 0, None) == 1
    for args, want in [((-1, 10, 0), 5), ((4, 0, 0), 5), ((4, 10, -1), 5), ((1 << 23, 10, 0), 3), ((4, 1 << 31, 0), 3),
                       ((4, 10, 1 << 23), 3), ((0, 10, 0), 0)]:
        assert f(*args, ctypes.byref(out)) == want, args
    assert out.value == 0


class _Call:
    """A valid call's arguments, to be spoilt one at a time."""

    def __init__(self, ah, pairs):
        self.ah, self.pairs = ah, pairs
        self.Y = ah.ArcheadTensor(FAKE, N, V, V, ah.ARCHEAD_BF16)
        self.dY = ah.ArcheadTensor(FAKE + (1 << 28), N, V, V, ah.ARCHEAD_F32)
        p = [FAKE + (2 << 28) + 4096 * i for i in range(12)]
        if pairs:
            self.inp = ah.ArcheadPreferenceInputs(p[0], p[1], 2, p[2], p[3], p[4], 0.1, 0.0, 1.0, 0)
            self.out = ah.ArcheadPreferenceOutputs(p[5], p[6], p[7], p[8], ctypes.pointer(self.dY))
        else:
            self.inp = ah.ArcheadPolicyInputs(p[0], p[1], p[2], p[3], p[4], 0.2, 0.2, 0.1, 1.0)
            self.out = ah.ArcheadPolicyOutputs(p[5], p[6], p[7], ctypes.pointer(self.dY))
        self.ws, self.ws_bytes = FAKE + (3 << 28), ah.archead_loss_workspace_bytes(N, V, 2 if pairs else 0)

    def __call__(self, null=None):
        f = self.ah.lib.archead_preference_loss if self.pairs else self.ah.lib.archead_policy_loss
        refs = [ctypes.byref(x) for x in (self.Y, self.inp, self.out)]
        if null is not None:
            refs[null] = None
        return f(*refs, self.ws, self.ws_bytes, None)


COMMON = [
    ("Y.dtype", 9, 4), ("dY.dtype", 0, 4), ("Y.cols", 0, 5), ("Y.rows", -1, 5), ("Y.row_stride", V - 1, 5),
    ("dY.rows", N - 1, 5), ("dY.cols", V + 1, 5), ("dY.row_stride", V - 1, 5), ("inp.inv_temperature", 0.0, 9),
    ("inp.inv_temperature", -1.0, 9), ("inp.inv_temperature", float("nan"), 9), ("inp.inv_temperature", float("inf"), 9),
    ("inp.labels", None, 1), ("Y.data", None, 1), ("dY.data", None, 1), ("Y.data", FAKE + 1, 6),
    ("dY.data", FAKE + (1 << 28) + 2, 6), ("inp.labels", FAKE + 2, 6), ("inp.weight", FAKE + 1, 6),
    ("out.loss", FAKE + 2, 6), ("out.logp", FAKE + 3, 6), ("ws", None, 1), ("ws", FAKE + 128, 6), ("ws_bytes", 255, 7),
    ("dY.data", FAKE + 4, 5), ("dY.data", FAKE, 5),  # over Y, but not Y itself
]
POLICY = [("inp.clip_low", -0.1, 9), ("inp.clip_high", float("nan"), 9), ("inp.kl_coef", -1.0, 9),
          ("inp.kl_coef", float("inf"), 9), ("inp.advantage", None, 1), ("inp.ref_logp", None, 1),
          ("inp.old_logp", FAKE + 2, 6), ("out.row_loss", FAKE + 2, 6)]
PREFERENCE = [("inp.offsets", None, 1), ("inp.offsets", FAKE + 2, 6), ("inp.n_pairs", -1, 5), ("inp.n_pairs", 1 << 23, 3),
              ("inp.kind", 2, 3), ("inp.kind", -1, 3), ("inp.beta", 0.0, 9), ("inp.beta", float("inf"), 9),
              ("inp.label_smoothing", 0.5, 9), ("inp.label_smoothing", -0.1, 9), ("inp.pair_weight", FAKE + 1, 6),
              ("out.chosen_reward", FAKE + 2, 6), ("out.rejected_reward", FAKE + 1, 6)]


@pytest.mark.parametrize("pairs,what,value,status", [(p, *c) for p, own in ((False, POLICY), (True, PREFERENCE))
                                                     for c in COMMON + own])
def test_loss_error_paths(ah, pairs, what, value, status):  # noqa: F811
    call = _Call(ah, pairs)
    *path, name = what.split(".")
    setattr(getattr(call, path[0]) if path else call, name, value)
    assert call() == status


@pytest.mark.parametrize("pairs", [False, True])
def test_loss_null_structs_and_empty_calls(ah, pairs):  # noqa: F811
    for i in range(3):
        assert _Call(ah, pairs)(null=i) == 1
    call = _Call(ah, pairs)  # no rows and no output: nothing to do, nothing needed
    call.Y.rows = call.dY.rows = 0
    call.Y.data = call.dY.data = call.inp.labels = call.out.loss = None
    if pairs:
        call.inp.n_pairs = 0
    call.ws, call.ws_bytes = None, 0
    assert call() == 0


def test_column_windows_of_one_buffer_do_not_overlap(ah):  # noqa: F811
    """dY in the right half of the rows whose left half is Y passes the overlap
    check (the call then fails at the workspace); one column further left it
    does not."""
    call = _Call(ah, False)
    call.dY.dtype = ah.ARCHEAD_BF16
    call.Y.row_stride = call.dY.row_stride = 2 * V
    call.ws_bytes = 0
    call.dY.data = FAKE + 2 * V
    assert call() == 7
    call.dY.data = FAKE + 2 * V - 2
    assert call() == 5
    call.dY.data, call.Y.data = FAKE, FAKE + 2 * V
    assert call() == 7
