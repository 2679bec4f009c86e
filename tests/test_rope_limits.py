"""Pairs on either side of the ramps of scaled rotary frequencies (host arithmetic)."""
import ctypes
import math

import pytest

import quantized_attention_diffusion_gb300 as qad
from quantized_attention_diffusion_gb300 import build as qbuild

YARN, BANDS = 3, 4


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qad.load_library()


@pytest.mark.parametrize("scaling", [YARN, BANDS])
@pytest.mark.parametrize("low,high", [(1.0, 32.0), (1.0, 4.0), (4.0, 40.0)])
@pytest.mark.parametrize("length", [1, 3, 6, 6.28, 6.29, 20, 25.1, 25.2, 100, 8192, 1e6, 1e9])
@pytest.mark.parametrize("dim", [2, 16, 128])
def test_pairs_outside_the_ramp(lib, dim, length, low, high, scaling):
    """Those that turn `high` times or more in the original length stay, those that turn `low`
    times or less are divided by the factor, the others are in between and no faster pair is
    divided by more."""
    f, plain, factor = (ctypes.c_uint64 * (dim // 2))(), (ctypes.c_uint64 * (dim // 2))(), ctypes.c_double()
    assert lib.sage_rope_frequencies(dim, 1e4, scaling, 4.0, float(length), low, high, f, ctypes.byref(factor)) == 0
    assert lib.sage_rope_frequencies(dim, 1e4, 0, 1.0, 1.0, 1.0, 2.0, plain, ctypes.byref(factor)) == 0
    last = 1.0 + 1e-9
    for i in range(dim // 2):
        turns, ratio = length * 1e4 ** (-2 * i / dim) / (2 * math.pi), f[i] / plain[i]
        if turns <= low * (1 - 1e-9):
            assert abs(ratio - 0.25) < 1e-9, i
        elif turns >= high * (1 + 1e-9):
            assert abs(ratio - 1.0) < 1e-9, i
        assert 0.25 - 1e-9 < ratio <= last
        last = ratio + 1e-9
