"""Outputs of the block operators that overlap what a call still reads: refused before any launch (no GPU
is touched; addresses are never dereferenced)."""
import ctypes

import pytest

FAKE = 1 << 20
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    import os
    from gated_delta_rule_69_amd import _block, _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gated_delta_rule_69_amd import build
        build.build()
    return _block._library()


def _conv(**over):
    from gated_delta_rule_69_amd._block import GdnConvArgs
    return ctypes.byref(GdnConvArgs(**{**dict(dtype=1, activation=1, B=2, T=100, C=64, W=4, x=FAKE, w=64 * FAKE, y=2 * FAKE), **over}))


ROWS = 2 * 100 * 64 * 2   # bytes of a contiguous [2, 100, 64] of bf16


@pytest.mark.parametrize("over", [
    dict(y=FAKE), dict(y=FAKE + 128), dict(y=FAKE - 128), dict(y=FAKE + ROWS - 128), dict(y=FAKE - ROWS + 128),
    dict(y=FAKE, T=9), dict(y=FAKE, x_stride=128), dict(y=FAKE, x_stride=128, T=1, B=3), dict(y=FAKE + 128, T=2),
    dict(y=FAKE + 128, x_stride=128), dict(y=FAKE - ROWS + 16, x_stride=128),
    dict(y=FAKE, dtype=0), dict(y=FAKE + 199 * 1024 + 112, x_stride=512)])
def test_convolution_over_its_own_input(lib, over):
    assert lib.gdn_short_conv_fwd(_conv(**over), None) == -1
    assert lib.gdn_short_conv_step(_conv(**over), 32 * FAKE, None) == -1
