"""Argument checks and workspace sizes of archead_cross_entropy (no GPU: every
call ends before the first HIP call)."""
import ctypes
import types

import pytest

from tests.test_abi import ah  # noqa: F401

FAKE = 1 << 30
STEP = 1 << 28
DIMS = (1024, 256, 16, 8, 64)


class _Call:
    def __init__(self, ah, dims=DIMS, fmt=0, n=40):  # noqa: F811
        V, D = dims[:2]
        self.ah, self.n, self.D = ah, n, D
        self.H = ah.ArcheadTensor(FAKE, n, D, D, ah.ARCHEAD_BF16)
        self.dH = ah.ArcheadTensor(FAKE + STEP, n, D, D, ah.ARCHEAD_BF16)
        self.P = ah.ArcheadPackedHead(ah.ArcheadDims(*dims, fmt), FAKE + 2 * STEP, 1 << 40, FAKE + 8 * STEP, 1 << 40)
        self.inp = ah.ArcheadCrossEntropyInputs(FAKE + 4 * STEP, FAKE + 5 * STEP, 1.0)
        self.out = ah.ArcheadCrossEntropyOutputs(FAKE + 6 * STEP, FAKE + 7 * STEP, None)
        self.gradient = True

    def __call__(self):
        self.out.dH = ctypes.pointer(self.dH) if self.gradient else None
        return self.ah.lib.archead_cross_entropy(ctypes.byref(self.H), ctypes.byref(self.P), ctypes.byref(self.inp),
                                                 ctypes.byref(self.out), None)


@pytest.mark.parametrize("n", [4, 40, 300])
@pytest.mark.parametrize("what,field,value,status", [
    ("H", "dtype", 2, 4), ("dH", "dtype", 2, 4), ("H", "cols", 255, 5), ("H", "row_stride", 248, 5), ("H", "rows", -1, 5),
    ("dH", "rows", 3, 5), ("dH", "cols", 257, 5), ("dH", "row_stride", 255, 5), ("H", "data", None, 1),
    ("dH", "data", None, 1), ("P", "buffer", None, 1), ("P", "workspace", None, 1), ("inp", "labels", None, 1),
    ("H", "data", FAKE + 8, 6), ("H", "row_stride", 260, 6), ("dH", "data", FAKE + STEP + 1, 6),
    ("inp", "labels", FAKE + 4 * STEP + 2, 6), ("inp", "weight", FAKE + 5 * STEP + 1, 6), ("out", "loss", FAKE + 2, 6),
    ("out", "logp", FAKE + 2, 6), ("P", "buffer", FAKE + 2 * STEP + 64, 6), ("P", "workspace", FAKE + 8 * STEP + 64, 6),
    ("P", "buffer_bytes", 1000, 10), ("P", "workspace_bytes", 1000, 7), ("inp", "inv_temperature", 0.0, 9),
    ("inp", "inv_temperature", -1.0, 9), ("inp", "inv_temperature", float("nan"), 9),
    ("inp", "inv_temperature", float("inf"), 9)])
def test_each_argument_is_checked(ah, n, what, field, value, status):  # noqa: F811
    call = _Call(ah, n=n)
    setattr(getattr(call, what), field, value)
    assert call() == status


@pytest.mark.parametrize("dims,fmt,n,status", [
    ((1024, 256, 0, 0, 64), 1, 4, 3), ((1024, 256, 0, 0, 64), 2, 4, 3), (DIMS, 3, 4, 2), ((1024, 256, 12, 8, 64), 0, 4, 3),
    ((1024, 256, 16, 8, 16), 0, 4, 3), ((1024, 200, 0, 0, 8), 0, 4, 2), (((1 << 24) + 1, 256, 16, 8, 64), 0, 4, 3),
    ((1024, 256, 1024, 8, 64), 0, 4, 3), (DIMS, 0, (1 << 22) + 1, 3),
    ((1024, 8192, 0, 0, 32), 0, 40, 3),   # 256 groups a row: no path of the forward takes 40 rows
])
def test_heads_that_are_not_served(ah, dims, fmt, n, status):  # noqa: F811
    assert _Call(ah, dims, fmt, n)() == status


@pytest.mark.parametrize("n", [4, 300])
def test_what_is_written_shares_no_bytes(ah, n):  # noqa: F811
    end = 2 * n * 256 - 4  # the last element of H or dH
    places = dict(H=FAKE + end, dH=FAKE + STEP + end, labels=FAKE + 4 * STEP + 4 * n - 4, weight=FAKE + 5 * STEP + 4 * n - 4,
                  head=FAKE + 2 * STEP + 512, ws=FAKE + 8 * STEP + 256, loss=FAKE + 6 * STEP, logp=FAKE + 7 * STEP + 4 * n - 4)
    for out in ("loss", "logp"):
        for other, at in places.items():
            if other != out:
                call = _Call(ah, n=n)
                setattr(call.out, out, at)
                assert call() == 5, (out, other)
    for other, at in places.items():
        call = _Call(ah, n=n)
        call.P.workspace = at // 256 * 256
        if other != "ws":
            assert call() == 5, ("ws", other)
        if other not in ("dH", "ws"):
            call = _Call(ah, n=n)
            call.dH.data = at
            assert call() == 5, ("dH", other)
    # column windows of rows of one buffer do not meet: the next check answers
    call = _Call(ah, n=n)
    call.H.row_stride = call.dH.row_stride = 1024
    call.dH.data = FAKE + 512
    call.out.loss = call.inp.labels
    assert call() == 5
    call.out.loss = FAKE + 6 * STEP
    call.dH.data = FAKE + 510
    assert call() == 5


def test_no_rows_null_structs_and_workspace(ah):  # noqa: F811
    call = _Call(ah, n=0)
    call.H.data = call.dH.data = call.P.buffer = call.P.workspace = call.inp.labels = call.inp.weight = None
    call.out.loss = call.out.logp = None
    assert call() == 0
    call = _Call(ah)
    args = [ctypes.byref(call.H), ctypes.byref(call.P), ctypes.byref(call.inp), ctypes.byref(call.out), None]
    for i in range(4):
        assert ah.lib.archead_cross_entropy(*args[:i], None, *args[i + 1:]) == 1
    f = ah.archead_cross_entropy_workspace_bytes
    assert f(*DIMS, 0) == 0
    big = (151936, 4096, 64, 64, 128)
    for dims in (DIMS, big, (33, 128, 0, 0, 32)):
        assert all(f(*dims, n) % 256 == 0 and f(*dims, n) > 0 for n in (1, 31, 32, 33, 64, 65, 4096, 4097))
    assert f(*big, 4096) < 4096 * 151936 * 2  # the logits alone in bf16 are more
    out = ctypes.c_uint64()
    g = ah.lib.archead_cross_entropy_workspace_bytes
    d = ah.ArcheadDims(*DIMS)
    assert g(None, 4, ctypes.byref(out)) == 1 and g(ctypes.byref(d), 4, None) == 1
    assert g(ctypes.byref(d), -1, ctypes.byref(out)) == 5 and g(ctypes.byref(d), 1 << 23, ctypes.byref(out)) == 3
    assert g(ctypes.byref(ah.ArcheadDims(1024, 256, 0, 0, 64, 2)), 4, ctypes.byref(out)) == 3


def test_a_stream_of_another_device_is_refused(ah):  # noqa: F811
    torch = pytest.importorskip("torch")
    first = types.SimpleNamespace(device=torch.device("cuda", 0))
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        ah.archead_cross_entropy(first, None, None, stream=stream)
