"""The products in 8-bit floats against the oracle: codes and exponents bit by bit, products within
the arithmetic of their sums.

Tolerance of a product, element by element, with mag the sum of the products' magnitudes: fp32
results sum exact products, one rounding (2^-24 of the partial sums, at most mag) for each of at most
ld / 8 + 8 additions; 16-bit results come from an instruction that aligns 64 products to the largest
and keeps at least 18 bits below it (each of 64 loses at most 2^-18 of the largest: 2^-12 mag), and
round once (half a step).  Sums over many products lose far less, since what is cut off has no
direction: relative to the norm at most 2e-4."""
import copy

import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from oracle import fp8 as of
from parity import TORCH_DT, say, to_np

pytestmark = pytest.mark.gpu


def tensors(m, n, k, cd, seed, bias=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))
    x[:, torch.randperm(k, generator=g)[: max(1, k // 150)]] *= 15
    w = torch.randn(n, k, generator=g) * 0.02
    b = torch.randn(n, generator=g).to(TORCH_DT[cd]) if bias else None
    return x.to(TORCH_DT[cd]), w.to(TORCH_DT[cd]), b


def check(y, ref, mag, cd, k, what=""):
    t = TORCH_DT[cd]
    got = to_np(y).astype(np.float64)
    lost = (k / 8 + 24) * 2.0 ** -24 if cd == "f32" else 2.0 ** -12
    tol = 1.1 * (lost * mag + torch.finfo(t).eps / 2 * np.abs(ref)) + float(torch.finfo(t).tiny) * torch.finfo(t).eps
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, first at %s: %r, expected %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0])
    if ref.size >= 64:
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= (1e-5 if cd == "f32" else 2e-4 + torch.finfo(t).eps / 2), "%s: rel %.2e" % (what, rel)


def same_codes(q, w):
    codes, scale = of.to_fp8(to_np(w), of.BLOCK)
    rows, cols = w.shape
    assert np.array_equal(to_np(q.codes), codes)
    kb = scale.shape[1]
    assert np.array_equal(to_np(q.scale)[:, :kb], scale) and (to_np(q.scale)[:, kb:] == 127).all()


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (128, 128), (129, 129), (130, 513), (300, 1000), (5, 131072)])
def test_weight_codes(rows, cols, cd):
    say("fp8 codes", rows, cols, cd)
    _, w, _ = tensors(1, rows, cols, cd, rows + cols)
    same_codes(qn.quantize_fp8(w.cuda()), w)


def test_weight_codes_at_edges():
    say("fp8 codes: edges")
    w = torch.zeros(8 * 128, 200)
    mid = torch.from_numpy((of.values()[:126] + of.values()[1:127]) / 2).float()
    w[0, 0], w[0, 1:127] = 448.0, mid                       # ties, scale 1
    w[128, 0], w[128, 1:127] = 448.0, torch.nextafter(mid, mid * 2)
    w[256, 0], w[256, 1:127] = -448.0, -torch.nextafter(mid, mid * 0)
    w[384, 5], w[385, 6] = 3.4028234e38, 1e30
    w[512, 3], w[513, 150] = float("inf"), 2.0
    w[640, 199], w[641, 0] = float("nan"), 1.0
    w[768, 0], w[769, 1] = 2.0 ** -130, -(2.0 ** -149)      # subnormal numbers
    w[896, :200] = torch.linspace(-1.7500001, 1.75, 200)
    same_codes(qn.quantize_fp8(w.cuda()), w)


def test_strided_weights_and_copies():
    say("fp8: strided weights")
    base = torch.randn(140, 177).cuda()
    for view in (base[:, 3:160], base[::2, :64], base.t(), base[:, 1:2], base[1:2, 2:9]):
        same_codes(qn.quantize_fp8(view), view.cpu())
    q = qn.quantize_fp8(base)
    x = torch.randn(3, 177).cuda()
    y = qn.linear_fp8(q, x)
    assert torch.equal(qn.linear_fp8(copy.deepcopy(q), x), y)
    q.codes = qn.quantize_fp8(base * 2 + 1).codes
    assert not torch.equal(qn.linear_fp8(q, x), y)
    q.rows = 139
    with pytest.raises(ValueError):
        qn.linear_fp8(q, x)
    assert qn.quantize_fp8(base[:0]).codes.shape == (0, 256)


SIZES = [(1, 1, 1), (1, 17, 64), (2, 64, 100), (5, 1000, 129), (16, 512, 1024), (17, 130, 4096), (33, 96, 300),
         (64, 257, 2048), (65, 128, 128), (128, 128, 256), (100, 1003, 511), (255, 300, 777), (256, 512, 1024),
         (300, 1030, 2047), (513, 640, 384), (1, 4096, 4096), (16, 14336, 512), (3, 200, 14336), (1030, 1290, 640),
         (1, 40, 16400), (1, 300, 131000), (15, 9000, 130), (300, 4099, 129), (520, 3001, 257), (2049, 2051, 130),
         (61, 500, 9000), (700, 64, 3328), (600, 4321, 1100)]


@pytest.mark.parametrize("cd", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_products(m, n, k, cd):
    say("fp8 product", m, n, k, cd)
    bias = (m + n) % 2 == 0
    x, w, b = tensors(m, n, k, cd, m + n + k, bias)
    out = torch.full((m + 2, n), float("nan"), dtype=TORCH_DT[cd]).cuda()
    y = qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda(), bias=None if b is None else b.cuda(), out=out[1:m + 1])
    ref, mag = of.product(to_np(x), to_np(w), None if b is None else to_np(b))
    check(y, ref, mag, cd, k)
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all()


@pytest.mark.parametrize("cd", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 384), (7, 300, 384), (60, 300, 384), (300, 700, 384)])
def test_far_scales(m, n, k, cd):
    """Tokens and weights near the ends of fp32's range whose products lie inside it."""
    say("fp8: far scales", m, n, k, cd)
    x, w, _ = tensors(m, n, k, cd, m + n)
    x, w = x.float(), w.float()
    x[0::3] = x[0::3] / x[0::3].abs().amax(1, keepdim=True) * 3e38
    x[1::3] *= 1e-36
    x[2::3] = 0
    w = w * 1e-30
    w[128:256] = 0
    x, w = x.to(TORCH_DT[cd]), w.to(TORCH_DT[cd])
    y = qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda())
    ref, mag = of.product(to_np(x), to_np(w))
    ref[1::3] = np.where(np.abs(ref[1::3]) < 1e-36, 0, ref[1::3])   # 1e-66: below fp32's smallest number
    check(y, ref, mag, cd, k)
    w = (w.double() * 1e60).to(TORCH_DT[cd])                         # now the small tokens' products are ordinary
    y = qn.linear_fp8(qn.quantize_fp8(w.cuda()), x[1::3].cuda())
    ref, mag = of.product(to_np(x[1::3]), to_np(w))
    check(y, ref, mag, cd, k)


@pytest.mark.parametrize("m", [1, 5, 40, 300])
@pytest.mark.parametrize("cd", ["bf16", "f16", "f32"])
def test_infinities_and_nans(m, cd):
    say("fp8: infinities and NaN", m, cd)
    x, w, _ = tensors(m, 200, 300, cd, m)
    w[7, 290], w[130, 4] = float("nan"), float("inf")
    x[m - 1, 5] = float("inf")
    if m > 2:
        x[1, 299] = float("nan")
    y = to_np(qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda()))
    nan = np.zeros((m, 200), bool)
    nan[:, :128] = True   # the blocks of the weight's NaN and infinity
    nan[:, 128:] = True
    assert np.isnan(y[nan]).all()
    w = tensors(m, 200, 300, cd, m)[1]
    y = to_np(qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda()))
    rows = np.zeros(m, bool)
    rows[[m - 1] + ([1] if m > 2 else [])] = True
    assert np.isnan(y[rows]).all() and np.isfinite(y[~rows]).all()


def test_views_leading_dims_and_refusals():
    say("fp8: views")
    x, w, b = tensors(24, 140, 260, "bf16", 3, True)
    q, xd = qn.quantize_fp8(w.cuda()), x.cuda()
    y = qn.linear_fp8(q, xd)
    assert torch.equal(qn.linear_fp8(q, xd.view(2, 3, 4, 260)), y.view(2, 3, 4, 140))
    wide = torch.randn(24, 300).bfloat16().cuda()
    wide[:, 7:267] = xd
    assert torch.equal(qn.linear_fp8(q, wide[:, 7:267]), y)
    assert torch.equal(qn.linear_fp8(q, xd[::2]), y[::2])
    assert torch.equal(qn.linear_fp8(q, xd.t().contiguous().t()), y)
    assert qn.linear_fp8(q, xd[:0]).shape == (0, 140)
    both = torch.zeros(24 * 400, dtype=torch.bfloat16).cuda()
    for bad in (lambda: qn.linear_fp8(q, xd, bias=b), lambda: qn.linear_fp8(q, xd.double()),
                lambda: qn.linear_fp8(q, xd[:, :250]), lambda: qn.linear_fp8(q, xd, out=y.float()),
                lambda: qn.linear_fp8(q, both[:24 * 260].view(24, 260), out=both[100:100 + 24 * 140].view(24, 140)),
                lambda: qn.linear_fp8(q, xd, workspace=torch.empty(8, dtype=torch.uint8).cuda()),
                lambda: qn.quantize_fp8(torch.zeros(2, 131073).cuda())):
        with pytest.raises((ValueError, TypeError, qn.QloraError)):
            bad()


def test_streams_and_graphs():
    say("fp8: streams and graphs")
    x, w, b = tensors(70, 300, 700, "bf16", 9, True)
    q, xd, bd = qn.quantize_fp8(w.cuda()), x.cuda(), b.cuda()
    one = xd[:1].clone()
    want, want1 = qn.linear_fp8(q, xd, bias=bd), qn.linear_fp8(q, one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qn.linear_fp8(q, xd, bias=bd)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, y1 = qn.linear_fp8(q, xd, bias=bd), qn.linear_fp8(q, one)
    for i in range(4):
        new = (x * (i + 1)).cuda()
        xd.copy_(new)
        one.copy_(new[:1])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, qn.linear_fp8(q, new, bias=bd)) and torch.equal(y1, qn.linear_fp8(q, new[:1]))
    assert torch.equal(qn.linear_fp8(q, x.cuda(), bias=bd), want) and torch.equal(want1, qn.linear_fp8(q, x[:1].cuda()))
