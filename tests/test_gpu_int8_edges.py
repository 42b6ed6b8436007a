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
