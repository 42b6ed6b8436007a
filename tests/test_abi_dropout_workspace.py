"""Workspaces of the dropout calls on the host: a query, which does not know the block size, covers what the
call on a weight of any layout takes.  A call without a workspace is refused before anything is launched, and its
message says what its plan needs."""
import ctypes
import random
import re

import pytest

from bit_nf4_quantized_nibble_amd import _lib

FAKE = 0x7F0000000000
OPS = (0, 1)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def weight(rows, cols, block, group=0):
    scales = (None, FAKE, FAKE) if group else (FAKE, None, None)
    return _lib.QloraNf4(rows, cols, block, int(group > 0), group or 256, 0, FAKE, *scales)


def refused(lib, op, w, m, r, cd, flags=0, ws_bytes=0):
    """The bytes that the seeded call asks for when it is refused for its workspace."""
    d = ctypes.byref(w)
    if op == 0:
        status = lib.qlora_linear_fwd_dropout_seeded(d, FAKE, m, FAKE, FAKE, r, 16.0, flags, None, cd, FAKE, 0.1, FAKE, None,
                                                     FAKE, ws_bytes, None)
    else:
        status = lib.qlora_linear_bwd_dropout_seeded(d, FAKE, FAKE, m, FAKE, FAKE, r, 16.0, flags, cd, FAKE, 0.1, None, 0,
                                                     FAKE, FAKE, FAKE, FAKE, ws_bytes, None)
    assert status == -5
    return int(re.search(r"(\d+) required", lib.qlora_last_error().decode()).group(1))


def query(lib, op, w, m, r, cd, flags=_lib.QLORA_FLAG_DROPOUT):
    return lib.qlora_workspace_bytes(op | flags << 8, m, w.rows, w.cols, r, cd)


# Calls of a decodable weight that take more slices of partial sums than the copy of W~ they save:
# op, tokens, rows, cols, rank, type
SLICES = [(0, 256, 8192, 256, 16, 1), (0, 256, 10176, 384, 8, 1), (0, 200, 14336, 256, 16, 1), (0, 128, 14336, 64, 16, 0),
          (1, 200, 256, 8192, 16, 1), (1, 256, 8192, 1024, 64, 1), (1, 256, 320, 14272, 8, 2), (1, 256, 4096, 2048, 64, 1),
          (1, 256, 1536, 4096, 64, 1)]


@pytest.mark.parametrize("op,m,rows,cols,r,cd", SLICES)
@pytest.mark.parametrize("block,group", [(64, 0), (32, 256)])
def test_seeded_query_covers_a_weight_that_is_decoded(lib, op, m, rows, cols, r, cd, block, group):
    w = weight(rows, cols, block, group)
    need = refused(lib, op, w, m, r, cd)
    assert 0 < need <= query(lib, op, w, m, r, cd)
    # the fp32 sums of the product, in one slice or more, and those of its low-rank part
    assert need >= 2 * m * (cols if op else rows) * 4
    assert refused(lib, op, w, m, r, cd, ws_bytes=need - 1) == need


def test_seeded_query_covers_every_layout(lib):
    rng = random.Random(7)

    def size(lo, hi):
        v = int(round(lo * (hi / lo) ** rng.random()))
        return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.6 else v

    for i in range(20000):
        op, cd, r = rng.choice(OPS), rng.randrange(3), rng.choice((1, 4, 8, 16, 33, 64, 100, 128))
        m, rows, cols = size(1, 300), size(64, 28672), size(64, 28672)
        whole = [b for b in (32, 64, 96, 128, 256) if cols % b == 0]
        block = rng.choice(whole) if whole and rng.random() < 0.8 else 2
        rows += rows * cols % block
        w = weight(rows, cols, block, rng.choice((0, 0, 100, 256)))
        flags = rng.choice((0, 0, 0, 2, 4))
        need = refused(lib, op, w, m, r, cd, flags)
        assert 0 < need <= query(lib, op, w, m, r, cd, flags | _lib.QLORA_FLAG_DROPOUT), (op, m, rows, cols, r, cd, block, flags)


def stored(lib, op, w, m, r, cd, flags=0):
    """The bytes that the call with a stored mask asks for when it is refused for its workspace."""
    d = ctypes.byref(w)
    if op == 0:
        status = lib.qlora_linear_fwd_dropout(d, FAKE, m, FAKE, FAKE, r, 16.0, flags, None, cd, FAKE, 0.1, FAKE, None, FAKE, 0,
                                              None)
    else:
        status = lib.qlora_linear_bwd_dropout(d, FAKE, FAKE, m, FAKE, FAKE, r, 16.0, flags, cd, FAKE, 0.1, None, FAKE, FAKE,
                                              FAKE, FAKE, 0, None)
    assert status == -5
    return int(re.search(r"(\d+) required", lib.qlora_last_error().decode()).group(1))


@pytest.mark.parametrize("flags", [0, 2, 4])
def test_a_stored_mask_needs_what_its_own_pass_stages(lib, flags):
    """The layer's plan without dropout, x M and (backward) the zeros in dT's place; nothing of the seeded call's."""
    up = lambda v: (v + 255) // 256 * 256
    for m, rows, cols, r, cd in ((100, 4096, 4096, 16, 0), (70, 14336, 4096, 64, 1), (4096, 4096, 4096, 64, 0),
                                 (4096, 4096, 14336, 64, 1), (300, 1000, 704, 12, 2), (65, 77, 130, 5, 1)):
        w, es = weight(rows, cols, 2), 2 if cd else 4
        both = _lib.QLORA_FLAG_DROPOUT | _lib.QLORA_FLAG_STORED_MASK | flags
        assert stored(lib, 0, w, m, r, cd, flags) == query(lib, 0, w, m, r, cd, both) \
            == query(lib, 0, w, m, r, cd, flags) + up(m * cols * es)
        assert stored(lib, 1, w, m, r, cd, flags) == query(lib, 1, w, m, r, cd, both) \
            == query(lib, 1, w, m, r, cd, flags) + up(m * cols * es) + up(m * ((r + 7) // 8 * 8) * es)
        for op in OPS:
            assert query(lib, op, w, m, r, cd, both) <= query(lib, op, w, m, r, cd, flags | _lib.QLORA_FLAG_DROPOUT)


def test_the_stored_mask_s_flag_stands_beside_dropout_s(lib):
    for op in OPS:
        assert query(lib, op, weight(64, 64, 64), 100, 8, 1, _lib.QLORA_FLAG_STORED_MASK) == 0
    assert query(lib, 2, weight(64, 64, 64), 100, 8, 1, 24) == 0
