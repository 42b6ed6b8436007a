"""The products in 8-bit integers where their kernels must agree with each other, and where a
weight changes between calls."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from oracle import int8 as oi
from parity import TORCH_DT, say, to_np
from test_gpu_int8 import check, tensors

pytestmark = pytest.mark.gpu


def test_a_weight_whose_storage_is_replaced():
    say("replaced storage")
    a, b, x = torch.randn(70, 130).cuda(), torch.randn(70, 130).cuda(), torch.randn(3, 130).cuda()
    q, want = qn.quantize_int8(a), qn.quantize_int8(b)
    first = qn.linear_int8(q, x)
    assert q.descriptor().codes == q.codes.data_ptr()
    kept = q.codes.data, q.scale.data
    q.codes.data, q.scale.data = want.codes.clone(), want.scale.clone()
    assert q.descriptor().codes == q.codes.data_ptr() != kept[0].data_ptr()
    assert q.descriptor().scale == q.scale.data_ptr() != kept[1].data_ptr()
    assert torch.equal(qn.linear_int8(q, x), qn.linear_int8(want, x))
    q.codes.data, q.scale.data = kept
    assert torch.equal(qn.linear_int8(q, x), first)
    q.rows = 69
    with pytest.raises(ValueError):
        qn.linear_int8(q, x)


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,batches,bias", [
    (4131, 384, (1, 2, 16, 17, 60, 300, 600, 2049, 4153), True),   # few tokens; every tile, the largest in rounds
    (4131, 384, (1, 16, 40, 4153), False),
    (1003, 14336, (1, 4, 16, 100, 300, 2000, 3000), True),         # slices of the contraction
])
def test_a_token_has_the_same_bits_in_every_batch(n, k, batches, bias, cd):
    """The sums are exact and the scaling is the same arithmetic in every kernel: fp32, then one
    rounding into the type."""
    say("batches", n, k, cd, bias)
    x, w, b = tensors(max(batches), n, k, cd, n + k, bias=bias)
    q, xd = qn.quantize_int8(w.cuda()), x.cuda()
    bd = None if b is None else b.cuda()
    whole = qn.linear_int8(q, xd, bias=bd)
    for m in batches:
        y = qn.linear_int8(q, xd[:m], bias=bd)
        differ = (y != whole[:m]).sum().item()
        assert differ == 0, "%d of %d elements of a batch of %d" % (differ, y.numel(), m)


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
def test_experts_have_the_bits_of_the_single_product(cd):
    say("experts against the single product", cd)
    sizes = [3, 0, 40, 700, 1, 256]
    x, w, b = tensors(sum(sizes), 1030, 700, cd, 21, experts=len(sizes), bias=True)
    q = qn.quantize_int8(w.cuda())
    off = np.r_[0, np.cumsum(sizes)]
    y = qn.linear_int8_experts(q, x.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), bias=b.cuda())
    for e in range(len(sizes)):
        s = slice(off[e], off[e + 1])
        one = qn.linear_int8(qn.quantize_int8(w[e].cuda()), x[s].cuda(), bias=b[e].cuda())
        assert torch.equal(y[s], one), "expert %d" % e


@pytest.mark.parametrize("cd", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 384), (7, 300, 384), (60, 300, 384), (300, 4131, 384), (600, 4131, 384),
                                   (2049, 4131, 384), (4153, 4131, 384), (4, 500, 14336), (100, 1003, 14336),
                                   (300, 4096, 7168)])
def test_products_that_pass_the_range_on_the_way(m, n, k, cd):
    """Tokens near the type's largest value on weights near zero: sum * s leaves fp32's range, y
    does not.  Ordinary tokens and zeros stand among them."""
    say("far tokens", m, n, k, cd)
    x, w, b = tensors(m, n, k, cd, m + n, bias=True)
    w = (w.float() * 1e-31).to(w.dtype)
    w[3] = 0
    xf = x.float()
    xf[::2] = xf[::2] / xf[::2].abs().amax(1, keepdim=True) * 3e38
    xf[1::4] *= 1e30
    if m > 4:
        xf[4] = 0
    x = xf.to(x.dtype)
    assert not x.isinf().any()
    q = qn.quantize_int8(w.cuda())
    y = qn.linear_int8(q, x.cuda(), bias=b.cuda())
    at = np.r_[0:min(m, 40), max(0, m - 40):m]
    ref, mag = oi.product(to_np(x)[at], *oi.rows_to_int8(to_np(w)), to_np(b))
    assert np.abs(ref).max() > 1e6
    check(y[torch.from_numpy(at).cuda()], ref, mag, cd)
    e = qn.linear_int8_experts(qn.quantize_int8(w[None].cuda()), x.cuda(),
                               torch.tensor([0, m], dtype=torch.int32, device="cuda"), bias=b[None].cuda())
    assert torch.equal(e, y)


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
def test_large_prompt_with_bias_and_odd_rows(cd):
    """Several rounds of the largest tiles, the last one in halves: biases and scales handed from tile
    to tile, rows of y that start anywhere, columns behind the last whole 16 bytes."""
    m, n, k = 4096 + 57, 4096 + 35, 384
    say("large prompt", m, n, k, cd)
    x, w, b = tensors(m, n, k, cd, 15, bias=True)
    y = qn.linear_int8(qn.quantize_int8(w.cuda()), x.cuda(), bias=b.cuda())
    codes, scale = oi.rows_to_int8(to_np(w))
    rows = np.r_[0:20, 120:136, 250:262, 2040:2056, 3960:3975, m - 70:m]
    ref, mag = oi.product(to_np(x)[rows], codes, scale, to_np(b))
    check(y[torch.from_numpy(rows).cuda()], ref, mag, cd)
    cols = np.r_[0:5, n - 37:n]
    ref, mag = oi.product(to_np(x), codes[cols], scale[cols], to_np(b)[cols])
    check(y[:, torch.from_numpy(cols).cuda()], ref, mag, cd, "columns")


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
def test_experts_of_many_rows(cd):
    """The same by expert: uneven, hundreds of rows each on average, more than one round of tiles."""
    sizes, n, k, before, tail = [900, 1, 0, 513, 129, 1400, 256], 9001, 200, 5, 9
    say("experts of many rows", cd)
    m = before + sum(sizes) + tail
    x, w, b = tensors(m, n, k, cd, 16, experts=len(sizes), bias=True)
    off = np.r_[0, np.cumsum(sizes)] + before
    out = torch.full((m, n), 7.0, dtype=TORCH_DT[cd], device="cuda")
    y = qn.linear_int8_experts(qn.quantize_int8(w.cuda()), x.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"),
                               bias=b.cuda(), out=out)
    assert (y[:before] == 7.0).all() and (y[m - tail:] == 7.0).all()
    for e, s in enumerate(sizes):
        rows = np.unique(np.r_[0:min(s, 6), min(s, 126):min(s, 131), min(s, 254):min(s, 259), max(0, s - 5):s]).astype(int)
        if s == 0:
            continue
        codes, scale = oi.rows_to_int8(to_np(w[e]))
        ref, mag = oi.product(to_np(x)[off[e] + rows], codes, scale, to_np(b[e]))
        check(y[torch.from_numpy(off[e] + rows).cuda()], ref, mag, cd, "expert %d" % e)
        cols = np.r_[0:3, n - 11:n]
        ref, mag = oi.product(to_np(x)[off[e]:off[e + 1]], codes[cols], scale[cols], to_np(b[e])[cols])
        check(y[int(off[e]):int(off[e + 1])][:, torch.from_numpy(cols).cuda()], ref, mag, cd, "columns of expert %d" % e)
