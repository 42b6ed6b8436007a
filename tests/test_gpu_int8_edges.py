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
