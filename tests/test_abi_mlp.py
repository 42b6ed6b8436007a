"""C-ABI checks of the 8-bit floating-point product, the gated block and the seeded dropout that
need no GPU: invalid calls are refused on the host before anything is launched."""
import ctypes

import pytest

from bit_nf4_quantized_nibble_amd import _lib

OK, INVALID, SHAPE, DTYPE, UNSUP, WS = 0, -1, -2, -3, -4, -5
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


# ---------------------------------------------------------------------------- 8-bit floats
def fdesc(rows=64, cols=96, reserved=0, codes=FAKE, scale=FAKE):
    return _lib.QloraFp8(rows, cols, reserved, codes, scale)


def fp8(lib, d, x=FAKE, m=5, ldx=96, bias=None, cd=1, y=FAKE + (1 << 20), ws=FAKE, ws_bytes=1 << 40):
    return lib.qlora_fp8_linear(ctypes.byref(d), x, m, ldx, bias, cd, y, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(reserved=1), INVALID), (dict(codes=None), INVALID),
    (dict(scale=None), INVALID), (dict(codes=FAKE + 8), INVALID), (dict(scale=FAKE + 2), INVALID),
    (dict(cols=131073), UNSUP), (dict(rows=1 << 31), UNSUP),
])
def test_fp8_bad_weights(lib, kw, status):
    d = fdesc(**kw)
    assert lib.qlora_fp8_quantize(FAKE, max(d.cols, 0), 1, ctypes.byref(d), None) == status
    assert lib.qlora_last_error()
    assert fp8(lib, d, ldx=1 << 20) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(bias=FAKE + 1), INVALID), (dict(x=FAKE + 2, cd=0), INVALID), (dict(m=-1), SHAPE), (dict(ldx=95), SHAPE),
    (dict(cd=5), DTYPE), (dict(m=1 << 31), UNSUP), (dict(ws_bytes=64), WS), (dict(ws=None), WS),
    (dict(ws=FAKE + 128), WS), (dict(y=FAKE), INVALID), (dict(y=FAKE + 5 * 192 - 2), INVALID),
    (dict(y=FAKE - 5 * 128 + 2), INVALID), (dict(m=0, x=None, y=None, ws=None, ws_bytes=0), OK),
])
def test_fp8_refusals(lib, kw, status):
    assert fp8(lib, fdesc(), **kw) == status


def test_fp8_empty_and_quantize(lib):
    assert fp8(lib, fdesc(rows=0)) == SHAPE and fp8(lib, fdesc(cols=0)) == SHAPE
    b = ctypes.byref(fdesc())
    q = lib.qlora_fp8_quantize
    assert q(None, 96, 1, b, None) == INVALID and q(FAKE + 1, 96, 1, b, None) == INVALID
    assert q(FAKE, 95, 1, b, None) == SHAPE and q(FAKE, 96, 3, b, None) == DTYPE and q(FAKE, 96, 1, None, None) == INVALID
    for kw in (dict(rows=0, codes=None, scale=None), dict(cols=0, codes=None, scale=None)):
        assert q(None, 96, 1, ctypes.byref(fdesc(**kw)), None) == OK


def test_fp8_workspace(lib):
    q = lib.qlora_fp8_workspace_bytes
    d = ctypes.byref(fdesc())
    assert q(d, 5, 1) >= 5 * 128 + 5 and q(d, 5, 1) % 256 == 0 and q(d, 0, 1) >= 0
    assert q(d, -1, 1) == 0 and q(d, 1 << 31, 1) == 0 and q(d, 5, 4) == 0 and q(None, 5, 1) == 0


# -------------------------------------------------------------------------------- NF4 calls
def ndesc(rows=256, cols=64, bs=64, codes=FAKE, absmax=FAKE):
    return _lib.QloraNf4(rows, cols, bs, 0, 256, 0, codes, absmax, None, None)


class Gated:
    def __init__(self, lib, d0=None, d1=None, r=(8, 4), alpha=(16.0, 8.0)):
        self.lib, self.d = lib, [d0 or ndesc(), d1 or ndesc()]
        self.w = (ctypes.POINTER(_lib.QloraNf4) * 2)(*[ctypes.pointer(d) for d in self.d])
        self.r, self.alpha = (ctypes.c_int32 * 2)(*r), (ctypes.c_float * 2)(*alpha)

    def ptrs(self, v):
        return None if v is None else (ctypes.c_void_p * 2)(*v)

    def fwd(self, x=FAKE, m=100, a=(FAKE, FAKE), b=(FAKE, FAKE), flags=0, act=0, bias=None, cd=1, h=FAKE, pre=None, t=None,
            ws=FAKE, ws_bytes=1 << 40):
        return self.lib.qlora_linear_fwd_gated(self.w, x, m, self.ptrs(a), self.ptrs(b), self.r, self.alpha, flags, act,
                                               bias, cd, h, pre, self.ptrs(t), ws, ws_bytes, None)

    def bwd(self, x=FAKE, dh=FAKE, pre=FAKE, m=100, a=(FAKE, FAKE), b=(FAKE, FAKE), flags=0, act=0, cd=1, t=None, gd=0,
            dx=FAKE, da=(FAKE, FAKE), db=(FAKE, FAKE), ws=FAKE, ws_bytes=1 << 40):
        return self.lib.qlora_linear_bwd_gated(self.w, x, dh, pre, m, self.ptrs(a), self.ptrs(b), self.r, self.alpha,
                                               flags, act, cd, self.ptrs(t), gd, dx, self.ptrs(da), self.ptrs(db), ws,
                                               ws_bytes, None)


BOTH = [(dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(a=None), INVALID), (dict(a=(FAKE, None)), INVALID),
        (dict(b=(None, FAKE)), INVALID), (dict(a=(FAKE + 4, FAKE)), INVALID), (dict(m=-1), SHAPE), (dict(flags=2), INVALID),
        (dict(flags=8), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(cd=7), DTYPE),
        (dict(t=(FAKE + 4, None)), INVALID), (dict(pre=FAKE + 2), INVALID), (dict(ws_bytes=64), WS), (dict(ws=None), WS)]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(h=None), INVALID), (dict(h=FAKE + 8), INVALID),
                                              (dict(bias=FAKE + 2), INVALID), (dict(m=0, ws=None, ws_bytes=0), OK)])
def test_gated_forward_refusals(lib, kw, status):
    assert Gated(lib).fwd(**kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(dh=None), INVALID), (dict(pre=None), INVALID), (dict(dh=FAKE + 8), INVALID), (dict(dx=FAKE + 8), INVALID),
    (dict(da=None), INVALID), (dict(da=(FAKE, None)), INVALID), (dict(db=(FAKE + 4, FAKE)), INVALID), (dict(gd=2), DTYPE),
    (dict(gd=5), DTYPE), (dict(m=0), SHAPE)])
def test_gated_backward_refusals(lib, kw, status):
    assert Gated(lib).bwd(**kw) == status


def test_gated_shapes(lib):
    for f in ("fwd", "bwd"):
        assert getattr(Gated(lib, d1=ndesc(rows=128)), f)() == SHAPE
        assert getattr(Gated(lib, d1=ndesc(cols=128)), f)() == SHAPE
        assert getattr(Gated(lib, r=(0, 4)), f)() == INVALID
        assert getattr(Gated(lib, alpha=(1.0, float("inf"))), f)() == INVALID
        assert getattr(Gated(lib, d0=ndesc(codes=None)), f)() == INVALID
    assert lib.qlora_linear_fwd_gated(None, FAKE, 4, None, None, None, None, 0, 0, None, 1, FAKE, None, None, FAKE, 1 << 30,
                                      None) == INVALID


def test_gated_workspace(lib):
    g = Gated(lib)
    q = lambda op=0, m=100, cd=1, w=g.w: lib.qlora_gated_workspace_bytes(op, w, m, g.r, cd)
    for op in (0, 1):
        for m in (1, 100, 300, 5000):
            for cd in (0, 1, 2):
                assert q(op, m, cd) > 0 and q(op, m, cd) % 256 == 0
        assert q(op, 5000) > q(op, 300)
    assert q(2) == 0 and q(cd=9) == 0 and q(m=-1) == 0 and q(w=Gated(lib, d1=ndesc(rows=128)).w) == 0


def drop_fwd(lib, d=None, m=128, seed=FAKE, p=0.1, r=8, cd=1, y=FAKE, ws_bytes=1 << 40, flags=0):
    return lib.qlora_linear_fwd_dropout_seeded(ctypes.byref(d or ndesc()), FAKE, m, FAKE, FAKE, r, 16.0, flags, None, cd,
                                               seed, p, y, None, FAKE, ws_bytes, None)


def drop_bwd(lib, d=None, m=128, seed=FAKE, p=0.1, r=8, cd=1, gd=0, da=FAKE, ws_bytes=1 << 40, flags=0):
    return lib.qlora_linear_bwd_dropout_seeded(ctypes.byref(d or ndesc()), FAKE, FAKE, m, FAKE, FAKE, r, 16.0, flags, cd,
                                               seed, p, None, gd, FAKE, da, FAKE, FAKE, ws_bytes, None)


@pytest.mark.parametrize("call", [drop_fwd, drop_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(seed=None), INVALID), (dict(seed=FAKE + 4), INVALID), (dict(p=1.0), INVALID), (dict(p=-0.1), INVALID),
    (dict(p=float("nan")), INVALID), (dict(r=0), INVALID), (dict(cd=4), DTYPE), (dict(m=-1), SHAPE), (dict(m=1 << 32), UNSUP),
    (dict(ws_bytes=64), WS), (dict(flags=6), INVALID)])
def test_seeded_dropout_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.qlora_last_error()


def test_seeded_dropout_edges(lib):
    assert drop_fwd(lib, m=0) == OK and drop_bwd(lib, m=0) == SHAPE
    assert drop_fwd(lib, y=None) == INVALID and drop_bwd(lib, da=None) == INVALID and drop_bwd(lib, da=FAKE + 8) == INVALID
    assert drop_bwd(lib, gd=2) == DTYPE and drop_bwd(lib, gd=9) == DTYPE


def test_binding_refuses_cpu_tensors_and_bad_names():
    torch = pytest.importorskip("torch")
    import bit_nf4_quantized_nibble_amd as qn

    with pytest.raises(ValueError):
        qn.quantize_fp8(torch.zeros(4, 4))
    x = torch.zeros(2, 64)
    q = qn.NF4Weight(64, 64, 64, False, 256, torch.zeros(2048, dtype=torch.uint8), torch.zeros(64))
    a, b = torch.zeros(4, 64), torch.zeros(64, 4)
    for call in (lambda: qn.linear_fwd_gated((q, q), x, [a, a], [b, b], [1.0, 1.0]),
                 lambda: qn.linear_fwd_gated((q, q), x, [a, a], [b, b], [1.0, 1.0], act="relu"),
                 lambda: qn.linear_fwd_gated((q,), x, [a], [b], [1.0]),
                 lambda: qn.linear_fwd_dropout(q, x, a, b, 1.0, 0.1, torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


def test_workspace_queries_of_no_tokens(lib):
    """m = 0 (a call that does nothing) has a size too, for every layer call and type."""
    g = Gated(lib)
    for op in (0, 1):
        for cd in (0, 1, 2):
            for flags in (0, 2, 4, 8):
                lib.qlora_workspace_bytes(op | flags << 8, 0, 256, 64, 8, cd)
            lib.qlora_group_workspace_bytes(op, 2, g.w, 0, g.r, cd)
            lib.qlora_gated_workspace_bytes(op, g.w, 0, g.r, cd)
    for cd in (1, 2):
        lib.qlora_workspace_bytes(2, 0, 256, 64, 8, cd)


def test_operands_past_the_tiles_reach(lib):
    """A row so long that a tile's rows span 2^31 bytes is refused before anything is launched."""
    long = lambda cols: ndesc(rows=64, cols=cols)
    for cd, cols in ((0, 1 << 22), (1, 1 << 24)):
        g = Gated(lib, d0=long(cols), d1=long(cols))
        assert g.fwd(cd=cd, m=20 if cd == 0 else 200) == UNSUP and lib.qlora_last_error()
        assert g.bwd(cd=cd) == UNSUP
        assert drop_fwd(lib, d=long(cols), cd=cd) == UNSUP and drop_bwd(lib, d=long(cols), cd=cd) == UNSUP
        assert lib.qlora_gated_workspace_bytes(1, g.w, 100, g.r, cd) == 0
