"""Arithmetic of the exponents that the cross entropy's operands are taken
under, compiled for the CPU: whole numbers of any size in fp32, against exact
integers."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.conftest import ROOT

CXX = shutil.which("g++")
TOP = 14


@pytest.fixture(scope="module")
def exponent(tmp_path_factory):
    if CXX is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("exp")
    (d / "e.cpp").write_text('#include "exp_range.h"\n'
                             'extern "C" float exponent(float top, float ref) { return archead::exp_exponent(top, ref); }\n')
    lib = str(d / "e.so")
    subprocess.run([CXX, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", os.path.join(ROOT, "compressed_output_head_amd", "csrc"),
                    str(d / "e.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).exponent
    f.restype, f.argtypes = ctypes.c_float, [ctypes.c_float, ctypes.c_float]
    return f


def _whole():
    """Whole numbers of fp32 about every power of two, of both signs."""
    out = {0.0}
    for k in range(128):
        x = np.float32(2.0 ** k)
        for y in (x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))):
            y = np.float32(np.ceil(y))
            for _ in range(6):
                out |= {float(y), -float(y)}
                y = np.float32(max(np.ceil(np.nextafter(y, np.float32(np.inf))), y + np.float32(1)))
    return sorted(v for v in out if abs(v) < 3.4e38)


def test_a_rows_first_exponent(exponent):
    """Whole, and the largest operand is 2^14 exactly where fp32 can say it,
    else at most 2^15 (fp16 ends at 65504) and at least 1."""
    for top in _whole():
        E = exponent(top, -np.inf)
        assert E == int(E)
        operand = int(top) - int(E)
        exact = abs(int(top) - TOP) <= 2 ** 24
        assert operand == TOP if exact else 0 <= operand <= TOP + 1, (top, E)
        assert float(np.float32(top) - np.float32(E)) == operand  # what the kernel raises 2 to


def test_a_running_exponent_is_kept_or_left_as_the_exact_difference_says(exponent):
    for ref in _whole():
        near = {ref + d for d in (-1e6, -100, -1, 0, 1, 13, 14, 15, 16, 17, 18, 32, 1000)}
        for top in near | {float(np.nextafter(np.float32(ref), np.float32(np.inf))), -ref, 2 * ref}:
            with np.errstate(over="ignore"):
                top = float(np.float32(top))
            if top != np.ceil(top) or not np.isfinite(top):
                continue
            keep = int(top) - int(ref) <= TOP + 1
            E = exponent(top, ref)
            assert E == (ref if keep else exponent(top, -np.inf)), (top, ref)


def test_what_is_not_a_number(exponent):
    inf, nan = float("inf"), float("nan")
    assert exponent(-inf, -inf) == -inf  # no entry so far
    assert exponent(-inf, 3.0) == 3.0
    assert exponent(inf, 3.0) == inf and exponent(inf, -inf) == inf and exponent(inf, inf) == inf
    assert exponent(3.0, inf) == inf  # a row that is not finite stays so
    assert np.isnan(exponent(nan, 3.0)) and np.isnan(exponent(nan, -inf))
