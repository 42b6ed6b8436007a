"""The 8-bit floating-point product of a weight with more rows than one launch takes: refused on the host, ahead of
the launch that brings the tokens to 8 bits (which would report a HIP error here, where there may be no device)."""
import ctypes

import pytest

from bit_nf4_quantized_nibble_amd import _lib

FAKE = 0x7F0000000000


@pytest.mark.parametrize("rows,cols,m,cd", [
    (1 << 29, 96, 5, 0), (1 << 29, 96, 16, 0), ((1 << 31) - 1, 128, 1, 0), (1 << 30, 4224, 9, 1), (1 << 29, 5000, 1, 2),
    (1 << 30, 96, 9, 1), ((1 << 31) - 1, 512, 17, 0)])
def test_more_rows_than_a_launch_takes(rows, cols, m, cd):
    lib = _lib.lib()
    d = _lib.QloraFp8(rows, cols, 0, FAKE, FAKE)
    y = FAKE + (1 << 40)
    assert lib.qlora_fp8_linear(ctypes.byref(d), FAKE, m, cols, None, cd, y, FAKE, 1 << 50, None) == -4
    assert b"tiles in one call" in lib.qlora_last_error()
