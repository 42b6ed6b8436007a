"""The product in 8-bit floats where test_gpu_fp8.py does not go: a weight of which one block of rows is no number, and
arrays past 2^31 elements.  Tolerances are test_gpu_fp8.py's."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from oracle import fp8 as of
from parity import TORCH_DT, say, to_np
from test_gpu_fp8 import check, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 5, 40, 300])
@pytest.mark.parametrize("cd", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_block_that_is_no_number_stays_alone(m, cd, bad):
    """The 128 rows of the weight's block are NaN; every other row is what it is without it."""
    say("fp8: one bad block", m, cd, bad)
    x, w, _ = tensors(m, 400, 300, cd, m)
    want = qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda())
    w[130, 290] = bad
    q = qn.quantize_fp8(w.cuda())
    y = qn.linear_fp8(q, x.cuda())
    inside = torch.arange(400) // 128 == 1
    assert torch.isnan(y[:, inside]).all() and torch.equal(y[:, ~inside], want[:, ~inside])
    assert torch.isfinite(want).all()


@pytest.mark.parametrize("m,n,k,cd", [(m, n, k, "bf16") for n, k in ((12225, 1153), (12224, 2048), (12290, 1024), (12300, 4100))
                                      for m in (4, 5, 11, 12, 16)]
                         + [(m, n, k, cd) for m in (5, 16, 17) for n, k, cd in ((2048, 8200, "f32"), (2049, 8200, "f16"))])
def test_each_side_of_the_few_token_rules(m, n, k, cd):
    say("fp8: few tokens", m, n, k, cd)
    x, w, b = tensors(m, n, k, cd, m + n, True)
    y = qn.linear_fp8(qn.quantize_fp8(w.cuda()), x.cuda(), bias=b.cuda())
    ref, mag = of.product(to_np(x), to_np(w), to_np(b))
    check(y, ref, mag, cd, k)


@pytest.mark.parametrize("m,n,k,cd", [((1 << 31) // 4096 + 300, 64, 4096, "bf16"), ((1 << 31) // 14400 + 300, 14400, 128, "bf16"),
                                      ((1 << 31) // 4096 + 300, 64, 4096, "f32"), ((1 << 31) // 14400 + 300, 14400, 128, "f32")])
def test_more_than_two_to_the_31st_elements(m, n, k, cd):
    say("fp8: large", m, n, k, cd)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda", dtype=TORCH_DT[cd])
    w = torch.randn(n, k, generator=g, device="cuda").mul_(0.02).to(TORCH_DT[cd])
    y = qn.linear_fp8(qn.quantize_fp8(w), x)
    at = torch.from_numpy(np.r_[0:4, m // 2:m // 2 + 4, m - 310:m - 290, m - 4:m]).cuda()
    ref, mag = of.product(to_np(x[at]), to_np(w))
    check(y[at], ref, mag, cd, k)
