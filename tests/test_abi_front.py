"""Argument checks and workspace sizes of the norm, its gradient and the INT8
product (no GPU: every call ends before the first HIP call)."""
import ctypes

import pytest

from tests.test_abi import ah  # noqa: F401

FAKE = 1 << 30
STEP = 1 << 28
N, D = 4, 96
BF16, F32, I8 = 1, 2, 3


def _tensors(ah, names, dtypes):  # noqa: F811
    return {k: ah.ArcheadTensor(FAKE + i * STEP, N, D, D, t) for i, (k, t) in enumerate(zip(names, dtypes))}


class _Norm:
    """A call that would be taken, but for what a test changes."""
    names = ("x", "residual", "sum", "h", "codes")

    def __init__(self, ah):  # noqa: F811
        self.ah, self.t = ah, _tensors(ah, self.names, (BF16, BF16, BF16, BF16, I8))
        self.v = dict(weight=FAKE + 8 * STEP, scale=FAKE + 9 * STEP, inv_rms=FAKE + 10 * STEP)
        self.eps = 1e-6

    def __call__(self):
        p = lambda k: ctypes.addressof(self.t[k]) if self.t[k] is not None else None  # noqa: E731
        inp = self.ah.ArcheadRmsnormInputs(p("x"), p("residual"), self.v["weight"], self.eps)
        out = self.ah.ArcheadRmsnormOutputs(p("sum"), p("h"), p("codes"), self.v["scale"], self.v["inv_rms"])
        return self.ah.lib.archead_rmsnorm(inp, out, None)


class _Grad(_Norm):
    names = ("dh", "sum", "dsum", "dx")

    def __init__(self, ah):  # noqa: F811
        self.ah, self.t = ah, _tensors(ah, self.names, (BF16,) * 4)
        self.v = dict(weight=FAKE + 8 * STEP, inv_rms=FAKE + 9 * STEP, dweight=FAKE + 10 * STEP, ws=FAKE + 11 * STEP)
        self.bytes = 1 << 20

    def __call__(self):
        p = lambda k: ctypes.addressof(self.t[k]) if self.t[k] is not None else None  # noqa: E731
        inp = self.ah.ArcheadRmsnormGradInputs(p("dh"), p("sum"), self.v["inv_rms"], self.v["weight"], p("dsum"))
        out = self.ah.ArcheadRmsnormGradOutputs(p("dx"), self.v["dweight"])
        return self.ah.lib.archead_rmsnorm_backward(inp, out, self.v["ws"], self.bytes, None)


@pytest.mark.parametrize("kind", [_Norm, _Grad])
def test_each_tensor_is_checked(ah, kind):  # noqa: F811
    for name in kind.names:
        changes = [("dtype", F32, 4), ("dtype", 0, 4), ("cols", D + 1, 5), ("row_stride", D - 1, 5), ("rows", N + 1, 5),
                   ("rows", -1, 5), ("data", None, 1)]
        if name != "codes":
            changes.append(("data", FAKE + 12 * STEP + 1, 6))
        for field, value, status in changes:
            call = kind(ah)
            setattr(call.t[name], field, value)
            assert call() == status, (name, field, value)


@pytest.mark.parametrize("kind", [_Norm, _Grad])
def test_sizes_that_are_not_served(ah, kind):  # noqa: F811
    for rows, cols, status in ((N, 32769, 3), ((1 << 22) + 1, D, 3), (N, 0, 5)):
        call = kind(ah)
        for t in call.t.values():
            t.rows, t.cols, t.row_stride = rows, cols, max(cols, 1)
        assert call() == status, (rows, cols)


def test_norm_scalars_and_vectors(ah):  # noqa: F811
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        call = _Norm(ah)
        call.eps = eps
        assert call() == 9
    for name, off in (("weight", 1), ("scale", 2), ("inv_rms", 2)):
        call = _Norm(ah)
        call.v[name] += off
        assert call() == 6, name
    call = _Norm(ah)
    call.v["scale"] = None  # codes without a scale
    assert call() == 1
    call = _Norm(ah)
    call.t["codes"] = None  # a scale without codes
    assert call() == 1
    call = _Norm(ah)
    for k in ("sum", "h", "codes"):
        call.t[k] = None
    call.v["scale"] = call.v["inv_rms"] = None
    assert call() == 0  # nothing is wanted
    assert ah.lib.archead_rmsnorm(None, None, None) == 1
    call = _Norm(ah)
    call.t["x"] = None
    assert call() == 1
    call = _Norm(ah)
    for t in call.t.values():
        t.rows, t.data = 0, None
    assert call() == 0


def _meets(call, out, other):
    """A tensor or vector `out` placed on `other`'s last byte."""
    size = {BF16: 2, I8: 1}
    if other in call.t:
        t = call.t[other]
        end = t.data + (N * D - 1) * size[t.dtype]
    else:
        end = call.v[other] + {"weight": 2 * D, "scale": 4 * N, "inv_rms": 4 * N, "dweight": 4 * D, "ws": 4 * D}[other] - 4
    if out in call.t:
        call.t[out].data = end // 2 * 2
    else:
        call.v[out] = end // 256 * 256 if out == "ws" else end // 4 * 4
    return call()


@pytest.mark.parametrize("kind,outs,ins", [
    (_Norm, ("sum", "h", "codes", "scale", "inv_rms"), ("x", "residual", "weight")),
    (_Grad, ("dx", "dweight", "ws"), ("dh", "sum", "dsum", "weight", "inv_rms"))])
def test_outputs_that_share_bytes_are_refused(ah, kind, outs, ins):  # noqa: F811
    for out in outs:
        for other in outs + ins:
            if other != out:
                assert _meets(kind(ah), out, other) == 5, (out, other)


def test_rows_that_may_be_replaced(ah):  # noqa: F811
    """In place the call goes on: the next check answers."""
    for out in ("sum", "h"):
        for name in ("x", "residual"):
            call = _Norm(ah)
            call.t[out].data = call.t[name].data
            call.t["codes"].data = call.v["weight"]  # refused last
            assert call() == 5
            call.t["codes"] = None
            call.v["scale"] = None
            call.t["sum" if out == "h" else "h"] = None
            call.t[out].row_stride = D + 2  # rows that wander over others
            assert call() == 5
    for name in ("dh", "sum", "dsum"):
        call = _Grad(ah)
        call.t["dx"].data = call.t[name].data + 2
        assert call() == 5
    call = _Norm(ah)  # codes never replace
    call.t["codes"].data = call.t["x"].data
    assert call() == 5


def test_gradient_vectors_and_workspace(ah):  # noqa: F811
    for name, off, status in (("weight", 1, 6), ("inv_rms", 2, 6), ("dweight", 2, 6), ("ws", 64, 6)):
        call = _Grad(ah)
        call.v[name] += off
        assert call() == status, name
    for name in ("inv_rms", "ws"):
        call = _Grad(ah)
        call.v[name] = None
        assert call() == 1
    call = _Grad(ah)
    call.bytes = ah.archead_rmsnorm_backward_workspace_bytes(N, D) - 1
    assert call() == 7
    call = _Grad(ah)
    call.t["dx"], call.v["dweight"] = None, None
    assert call() == 0
    for name in ("dh", "sum"):
        call = _Grad(ah)
        call.t[name] = None
        assert call() == 1
    f = ah.archead_rmsnorm_backward_workspace_bytes
    assert f(0, 5) == 0 and f(1, 1) == 256 and f(4096, 4096) % 256 == 0
    assert all(f(n, 1000) <= f(n + 1, 1000) for n in (1, 7, 100, 3000, 9999))
    out = ctypes.c_uint64()
    g = ah.lib.archead_rmsnorm_backward_workspace_bytes
    assert g(4, 4, None) == 1 and g(-1, 4, ctypes.byref(out)) == 5 and g(4, 0, ctypes.byref(out)) == 5
    assert g(1 << 23, 4, ctypes.byref(out)) == 3 and g(4, 1 << 16, ctypes.byref(out)) == 3


I8_DIMS = (1000, 256, 0, 0, 64)


def _int8(ah, dims=I8_DIMS, fmt=2, n=40, scale=FAKE + STEP, **kw):  # noqa: F811
    V, D = dims[:2]
    X = ah.ArcheadTensor(FAKE, n, D, D, I8)
    Y = ah.ArcheadTensor(FAKE + 2 * STEP, n, V, V, F32)
    P = ah.ArcheadPackedHead(ah.ArcheadDims(*dims, fmt), FAKE + 4 * STEP, 1 << 40, FAKE + 6 * STEP, 1 << 40)
    for k, v in kw.items():
        what, name = k.split("_", 1)
        setattr(dict(X=X, Y=Y, P=P)[what], name, v)
    return ah.lib.archead_logits_int8(ctypes.byref(X), scale, ctypes.byref(P), ctypes.byref(Y), None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=0), 3), (dict(fmt=1), 3), (dict(fmt=3), 2), (dict(dims=(1000, 200, 0, 0, 8)), 2),
    (dict(dims=(1000, 65536 + 128, 0, 0, 128)), 3), (dict(n=(1 << 22) + 1), 3), (dict(n=-1), 5),
    (dict(X_dtype=1), 4), (dict(Y_dtype=3), 4), (dict(X_cols=255), 5), (dict(X_row_stride=240), 5), (dict(Y_rows=39), 5),
    (dict(Y_cols=999), 5), (dict(Y_row_stride=999), 5), (dict(X_data=None), 1), (dict(Y_data=None), 1), (dict(scale=None), 1),
    (dict(P_buffer=None), 1), (dict(P_workspace=None), 1), (dict(X_data=FAKE + 8), 6), (dict(X_row_stride=264), 6),
    (dict(Y_data=FAKE + 2 * STEP + 2), 6), (dict(scale=FAKE + 2), 6), (dict(P_buffer=FAKE + 128), 6),
    (dict(P_workspace=FAKE + 64), 6), (dict(P_buffer_bytes=1000), 10), (dict(P_workspace_bytes=64 * 256 - 1), 7),
    # Y over X, the scales, the head and the workspace, and the calls next to those
    (dict(Y_data=FAKE + 40 * 256 - 4), 5), (dict(Y_data=FAKE + 40 * 256, P_workspace_bytes=0), 7),
    (dict(Y_data=FAKE - 160000 + 4), 5), (dict(Y_data=FAKE + STEP + 156), 5), (dict(Y_data=FAKE + 4 * STEP + 256), 5),
    (dict(Y_data=FAKE + 6 * STEP + 64 * 256 - 4), 5),
])
def test_int8_error_paths(ah, kw, status):  # noqa: F811
    assert _int8(ah, **kw) == status


def test_int8_no_rows_and_workspace(ah):  # noqa: F811
    assert _int8(ah, n=0, X_data=None, Y_data=None, P_buffer=None, P_workspace=None, scale=None) == 0
    f = ah.archead_logits_int8_workspace_bytes
    assert f(1000, 256, 64, 0) == 0 and f(1000, 256, 64, 8) == 0 and f(1000, 256, 64, 9) == 32 * 256
    assert f(1000, 32768, 64, 8) == 32 * 32768  # 8 rows of this size do not fit LDS
    assert f(1000, 256, 64, 1 << 20) == 16384 * 256
    out = ctypes.c_uint64()
    g = ah.lib.archead_logits_int8_workspace_bytes
    d = ah.ArcheadDims(*I8_DIMS, 2)
    assert g(None, 4, ctypes.byref(out)) == 1 and g(ctypes.byref(d), 4, None) == 1
    assert g(ctypes.byref(d), -1, ctypes.byref(out)) == 5 and g(ctypes.byref(d), 1 << 23, ctypes.byref(out)) == 3
    assert g(ctypes.byref(ah.ArcheadDims(*I8_DIMS, 0)), 4, ctypes.byref(out)) == 3
    t = ah.ArcheadTensor(FAKE, 4, 256, 256, 3)
    assert ah.lib.archead_logits_int8(None, FAKE, None, ctypes.byref(t), None) == 1


@pytest.mark.parametrize("name", ["archead_rmsnorm", "archead_rmsnorm_backward", "archead_logits_int8"])
def test_a_stream_of_another_device_is_refused(ah, name):  # noqa: F811
    import types
    torch = pytest.importorskip("torch")
    first = types.SimpleNamespace(device=torch.device("cuda", 0))
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        getattr(ah, name)(first, None, None, stream=stream)
