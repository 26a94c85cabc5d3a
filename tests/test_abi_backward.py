"""Argument checks and workspace sizes of archead_logits_backward (no GPU:
every call fails validation before the first HIP call)."""
import ctypes

import pytest

from tests.test_abi import ah  # noqa: F401

FAKE = 1 << 30
DIMS = (1024, 256, 16, 8, 64)


def _call(ah, dims=DIMS, fmt=0, N=4, **kw):
    V, D = dims[:2]
    dY = ah.ArcheadTensor(FAKE, N, V, V, ah.ARCHEAD_BF16)
    dH = ah.ArcheadTensor(FAKE + (1 << 28), N, D, D, ah.ARCHEAD_BF16)
    P = ah.ArcheadPackedHead(ah.ArcheadDims(*dims, fmt), FAKE + (2 << 28), 1 << 40, FAKE + (3 << 28), 1 << 40)
    for k, v in kw.items():
        what, name = k.split("_", 1)
        setattr(dict(dY=dY, dH=dH, P=P)[what], name, v)
    return ah.lib.archead_logits_backward(ctypes.byref(dY), ctypes.byref(P), ctypes.byref(dH), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dY_dtype=0), 4), (dict(dY_dtype=3), 4), (dict(dH_dtype=2), 4), (dict(dY_cols=1023), 5),
    (dict(dY_row_stride=1023), 5), (dict(dY_rows=-1), 5), (dict(dH_rows=3), 5), (dict(dH_cols=257), 5),
    (dict(dH_row_stride=255), 5), (dict(dY_data=None), 1), (dict(dH_data=None), 1), (dict(P_buffer=None), 1),
    (dict(P_workspace=None), 1), (dict(dY_data=FAKE + 1), 6), (dict(dH_data=FAKE + 1), 6),
    (dict(P_buffer=FAKE + 128), 6), (dict(P_workspace=FAKE + 16), 6), (dict(P_buffer_bytes=1000), 10),
    (dict(P_workspace_bytes=1000), 7), (dict(fmt=1, dims=(1024, 256, 0, 0, 64)), 3), (dict(fmt=3), 2),
    (dict(dims=(1024, 256, 16, 8, 16)), 3), (dict(dims=(1024, 256, 12, 8, 64)), 3), (dict(dims=(1024, 200, 0, 0, 8)), 2),
    (dict(dims=(1024, 256, 1024, 8, 64)), 3), (dict(N=1 << 23), 3),
    (dict(dims=((1 << 26) + 1, 256, 16, 8, 64)), 3),
    # dH in dY's rows, from before them into them, and behind dY but for its last row's last elements
    (dict(dH_data=FAKE + 4096), 5), (dict(dH_data=FAKE - 1024), 5), (dict(dH_data=FAKE + 8190), 5),
    # column windows of rows of one buffer do not meet: the next check answers
    (dict(dH_data=FAKE + 2048, dH_row_stride=2048, dY_row_stride=2048, P_workspace_bytes=1000), 7),
    (dict(dH_data=FAKE + 2046, dH_row_stride=2048, dY_row_stride=2048, P_workspace_bytes=1000), 5),
])
def test_backward_error_paths(ah, kw, status):  # noqa: F811
    assert _call(ah, **kw) == status


def test_backward_null_structs_and_no_rows(ah):  # noqa: F811
    t = ah.ArcheadTensor(FAKE, 4, 1024, 1024, 1)
    P = ah.ArcheadPackedHead(ah.ArcheadDims(*DIMS), FAKE, 1 << 40, FAKE, 1 << 40)
    f = ah.lib.archead_logits_backward
    assert f(None, ctypes.byref(P), ctypes.byref(t), None) == 1
    assert f(ctypes.byref(t), None, ctypes.byref(t), None) == 1
    assert f(ctypes.byref(t), ctypes.byref(P), None, None) == 1
    assert _call(ah, N=0, dY_data=None, dH_data=None, P_buffer=None, P_workspace=None) == 0


def test_backward_workspace(ah):  # noqa: F811
    f = ah.archead_logits_backward_workspace_bytes
    assert f(*DIMS, 0) == 0
    for dims in (DIMS, (151936, 4096, 64, 64, 128), (33, 128, 0, 0, 32)):
        sizes = [f(*dims, n) for n in (1, 31, 32, 33, 4096, 4097, 12288, 12289)]
        assert all(s % 256 == 0 for s in sizes) and sizes[0] >= 3 * dims[0] * 2 + dims[1] * 4
        assert sizes[3] >= 64 * dims[0] * 2 + 33 * dims[1] * 4
        assert max(sizes[5:]) <= 2 * sizes[4]  # rows are taken 4096 at a time
        assert f(*dims, 4096 + 200) >= f(*dims, 200)
    out = ctypes.c_uint64()
    g = ah.lib.archead_logits_backward_workspace_bytes
    assert g(None, 4, ctypes.byref(out)) == 1 and g(ctypes.byref(ah.ArcheadDims(*DIMS)), 4, None) == 1
    assert g(ctypes.byref(ah.ArcheadDims(*DIMS)), -1, ctypes.byref(out)) == 5
    assert g(ctypes.byref(ah.ArcheadDims(1024, 256, 0, 0, 64, 2)), 4, ctypes.byref(out)) == 3
    assert g(ctypes.byref(ah.ArcheadDims(0, 256, 0, 0, 64)), 4, ctypes.byref(out)) == 2
