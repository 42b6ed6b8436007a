"""C-ABI checks of the 8-bit products and the distillation loss that need no GPU: invalid calls
are refused on the host before anything is launched (the pointers are never dereferenced)."""
import ctypes

import pytest

from bit_nf4_quantized_nibble_amd import _lib

OK, INVALID, SHAPE, DTYPE, UNSUP, WS = 0, -1, -2, -3, -4, -5
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def desc(rows=64, cols=96, experts=1, reserved=0, codes=FAKE, scale=FAKE):
    return _lib.QloraInt8(rows, cols, experts, reserved, codes, scale)


BAD_WEIGHT = [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(experts=0), INVALID), (dict(experts=-2), INVALID),
    (dict(reserved=1), INVALID), (dict(codes=None), INVALID), (dict(scale=None), INVALID),
    (dict(codes=FAKE + 8), INVALID), (dict(scale=FAKE + 2), INVALID), (dict(cols=131073), UNSUP),
    (dict(rows=1 << 31), UNSUP), (dict(rows=1 << 61, experts=16), UNSUP), (dict(rows=1 << 27, experts=16), UNSUP),
]


@pytest.mark.parametrize("kw,status", BAD_WEIGHT)
def test_bad_weights(lib, kw, status):
    d = desc(**kw)
    assert lib.qlora_int8_quantize(FAKE, max(d.cols, 0), 1, ctypes.byref(d), None) == status
    assert lib.qlora_last_error()
    if d.experts == 1:
        assert lib.qlora_int8_linear(ctypes.byref(d), FAKE, 4, 1 << 20, None, 1, FAKE, FAKE, 1 << 40, None) == status
    assert lib.qlora_int8_linear_experts(ctypes.byref(d), FAKE, 4, 1 << 20, FAKE, None, 1, FAKE, FAKE, 1 << 40,
                                         None) == status


def test_quantize_refusals(lib):
    d = desc()
    b = ctypes.byref(d)
    assert lib.qlora_int8_quantize(None, 96, 1, b, None) == INVALID
    assert lib.qlora_int8_quantize(FAKE + 1, 96, 1, b, None) == INVALID
    assert lib.qlora_int8_quantize(FAKE + 2, 96, 0, b, None) == INVALID
    assert lib.qlora_int8_quantize(FAKE, 95, 1, b, None) == SHAPE
    assert lib.qlora_int8_quantize(FAKE, 96, 3, b, None) == DTYPE
    assert lib.qlora_int8_quantize(FAKE, 96, 1, None, None) == INVALID
    for kw in (dict(rows=0, codes=None, scale=None), dict(cols=0, codes=None, scale=None)):
        d = desc(**kw)
        assert lib.qlora_int8_quantize(None, 96, 1, ctypes.byref(d), None) == OK


def linear(lib, d, x=FAKE, m=5, ldx=96, bias=None, cd=1, y=FAKE, ws=FAKE, ws_bytes=1 << 40, offsets=FAKE,
           grouped=False):
    if grouped:
        return lib.qlora_int8_linear_experts(ctypes.byref(d), x, m, ldx, offsets, bias, cd, y, ws, ws_bytes, None)
    return lib.qlora_int8_linear(ctypes.byref(d), x, m, ldx, bias, cd, y, ws, ws_bytes, None)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(bias=FAKE + 1), INVALID), (dict(x=FAKE + 2, cd=0), INVALID), (dict(m=-1), SHAPE), (dict(ldx=95), SHAPE),
    (dict(cd=5), DTYPE), (dict(m=1 << 31), UNSUP), (dict(ws_bytes=64), WS), (dict(ws=None), WS),
    (dict(ws=FAKE + 128), WS),
])
def test_linear_refusals(lib, kw, status, grouped):
    assert linear(lib, desc(), grouped=grouped, **kw) == status
    assert lib.qlora_last_error()


def test_linear_shapes(lib):
    assert linear(lib, desc(rows=0)) == SHAPE
    assert linear(lib, desc(cols=0)) == SHAPE
    assert linear(lib, desc(experts=2)) == INVALID              # the form grouped by expert takes those
    assert linear(lib, desc(experts=2), grouped=True, offsets=None) == INVALID
    assert linear(lib, desc(experts=2), grouped=True, offsets=FAKE + 2) == INVALID
    assert linear(lib, desc(experts=65536), grouped=True) == UNSUP
    for grouped in (False, True):  # y over x: at its start, its last element, and x at y's last
        for m, y in ((5, FAKE), (5, FAKE + 5 * 192 - 2), (5, FAKE - 5 * 128 + 2), (1, FAKE + 190), (1, FAKE - 126)):
            assert linear(lib, desc(), m=m, y=y, grouped=grouped) == INVALID
            assert b"overlaps" in lib.qlora_last_error()
    assert linear(lib, desc(), m=0, x=None, y=None, ws=None, ws_bytes=0) == OK
    assert linear(lib, desc(experts=3), m=0, x=None, y=None, ws=None, ws_bytes=0, grouped=True) == OK


def test_int8_workspace_queries(lib):
    q = lib.qlora_int8_workspace_bytes
    d = desc(rows=100, cols=200, experts=4)
    assert q(ctypes.byref(d), 10, 0) == 0 and q(ctypes.byref(d), 10, 1) >= 10 * 256
    assert q(ctypes.byref(desc()), 10, 0) >= 10 * 128
    assert q(ctypes.byref(desc()), -1, 0) == 0 and q(None, 4, 0) == 0
    assert q(ctypes.byref(desc(codes=None, scale=None)), 4, 0) > 0  # shapes only
    for rows, cols in ((0, 96), (0, 14336), (0, 131072), (64, 0)):  # empty weights
        for m in (0, 1, 100, 5000):
            for grouped in (0, 1):
                assert q(ctypes.byref(desc(rows=rows, cols=cols)), m, grouped) <= m * (131072 + 4) + 100000


def distill(lib, z=FAKE, n=4, vocab=100, ld=100, cd=1, u=FAKE, td=0, idx=FAKE, bits=32, k=8, t=1.0, w=None, loss=FAKE,
            kl=None, dz=FAKE + 4096, ldd=100, ws=FAKE, ws_bytes=1 << 20):
    return lib.qlora_distill_loss_grad(z, n, vocab, ld, cd, u, td, idx, bits, k, t, w, loss, kl, dz, ldd, ws, ws_bytes,
                                       None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), INVALID), (dict(u=None), INVALID), (dict(idx=None), INVALID), (dict(loss=None), INVALID),
    (dict(z=FAKE + 1), INVALID), (dict(dz=FAKE + 4097), INVALID), (dict(u=FAKE + 2), INVALID),
    (dict(idx=FAKE + 4, bits=64), INVALID), (dict(w=FAKE + 2), INVALID), (dict(kl=FAKE + 1), INVALID),
    (dict(loss=FAKE + 2), INVALID), (dict(bits=16), INVALID), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID),
    (dict(t=float("nan")), INVALID), (dict(t=float("inf")), INVALID), (dict(t=9e-7), INVALID), (dict(t=2e6), INVALID), (dict(n=-1), SHAPE), (dict(vocab=0), SHAPE),
    (dict(k=0), SHAPE), (dict(ld=99), SHAPE), (dict(ldd=99), SHAPE), (dict(cd=3), DTYPE), (dict(td=-1), DTYPE),
    (dict(dz=FAKE + 200), INVALID), (dict(z=FAKE + 4296), INVALID), (dict(dz=FAKE, z=FAKE, ldd=108), INVALID),
    (dict(z=FAKE, dz=FAKE + 198, ld=200, ldd=200), INVALID), (dict(z=FAKE, dz=FAKE + 202, ld=200, ldd=200), INVALID),
    (dict(k=1025), UNSUP), (dict(n=1 << 31), UNSUP), (dict(vocab=1 << 31, ld=1 << 31, ldd=1 << 31), UNSUP),
    (dict(ws_bytes=8), WS), (dict(ws=FAKE + 64), WS), (dict(ws=None), WS),
])
def test_distill_refusals(lib, kw, status):
    assert distill(lib, **kw) == status
    assert lib.qlora_last_error()


def test_distill_workspace_queries(lib):
    q = lib.qlora_distill_workspace_bytes
    assert q(-1, 10, 1, 1) == 0 and q(0, 10, 1, 1) > 0 and q(1000, 10, 1, 1) >= 4000
    assert q(4, 0, 1, 1) == 0 and q(4, 10, 0, 1) == 0 and q(4, 10, 1025, 1) == 0 and q(4, 10, 1, 3) == 0
    assert q(4, 100000, 8, 1) > q(4, 100, 8, 1)  # rows cut into parts


def test_tiles_beyond_one_launch_are_refused_before_any_work(lib):
    """A launch has fewer than 2^32 threads: experts' tiles of more are refused on the host."""
    d = desc(rows=32000, cols=64, experts=65535)
    assert linear(lib, d, m=65535 * 60, grouped=True, ws_bytes=1 << 62, x=FAKE, y=FAKE + (1 << 40)) == UNSUP
    assert b"tiles" in lib.qlora_last_error()
    d = desc(rows=(1 << 31) - 1, cols=64)
    assert linear(lib, d, m=(1 << 31) - 1, ws_bytes=1 << 62, x=FAKE, y=FAKE + (1 << 40)) == UNSUP
    assert b"tiles" in lib.qlora_last_error()


def test_workspaces_hold_the_slices_only_where_the_contraction_is_cut(lib):
    def q(rows, cols, m, experts=1, grouped=0):
        return lib.qlora_int8_workspace_bytes(ctypes.byref(desc(rows=rows, cols=cols, experts=experts)), m, grouped)

    def tokens(cols, m):
        ld = (cols + 127) // 128 * 128
        return (m * ld + 255) // 256 * 256 + (4 * m + 255) // 256 * 256

    # one launch, or the few-token kernel: the tokens' codes and scales alone
    for rows, cols, m in ((4096, 14336, 1), (512, 16384, 1), (64, 32768, 1), (4096, 14336, 2), (4096, 14336, 16),
                          (4096, 4096, 16), (2049, 16384, 9)):
        assert q(rows, cols, m) == tokens(cols, m), (rows, cols, m)
    for m in (1, 8, 16):  # by expert: the run list besides
        assert q(2048, 14336, m, experts=4, grouped=1) <= tokens(14336, m) + 4096, m
    # slices of a long contraction
    for rows, cols, m in ((512, 16384, 16), (64, 131072, 1), (1000, 14336, 100), (4096, 14336, 300)):
        assert q(rows, cols, m) > tokens(cols, m) + 4 * rows * m, (rows, cols, m)
