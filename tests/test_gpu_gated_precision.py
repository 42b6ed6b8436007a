"""dA of the gated block's backward where it goes the general way: dT = s d B is the product of a sum whose terms may cancel,
so d goes into it as the sum of two 16-bit values.  What is left out of an element of d is at most u^2 = (eps / 2)^2 of it
(f16: or half of its smallest step), independent from element to element, so that dT is off by at most
s u^2 sqrt(sum_n d^2 B^2) in the mean square; four times that, and 1e-4 for dT's own two 16-bit parts, x's and the sums' fp32
and the activation's fp32, are the bound.  One rounding of d alone would be off by 1 / u = 256 (bf16) times as much."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from oracle import gated as og
from parity import TORCH_DT, say, to_np
from test_gpu_mlp_layouts import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,r,cd,block,group", [
    (1, 64, 65, 1, "bf16", 2, 0), (1, 64, 64, 1, "f16", 64, 0), (2, 4096, 64, 1, "bf16", 64, 256), (3, 128, 63, 7, "f16", 4, 256),
    (129, 96, 130, 80, "bf16", 96, 100), (257, 128, 256, 16, "bf16", 64, 0), (600, 2112, 100, 12, "bf16", 64, 0)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradient_of_a_small_sum(M, N, K, r, cd, block, group, act):
    say("gated dA", M, N, K, r, cd, block, group, act)
    (L0, o0, q0), (L1, o1, q1) = layer(M, N, K, r, cd, block, group, M), layer(M, N, K, r, cd, block, group, M + 1)
    x, dh = L0.x.cuda(), L0.dY.cuda()
    args = ((q0, q1), x, [L0.A.cuda(), L1.A.cuda()], [L0.B.cuda(), L1.B.cuda()], [L0.alpha, L1.alpha])
    _, pre, ts = qn.linear_fwd_gated(*args, act=act, save=True)
    _, da, _ = qn.linear_bwd_gated(args[0], x, dh, *args[2:], pre, act=act, t_saved=ts)
    p64 = to_np(pre).astype(np.float64)
    d = og.backward(p64[:, :N], p64[:, N:], o0["dY"], act)
    u = torch.finfo(TORCH_DT[cd]).eps / 2
    for i, o in enumerate((o0, o1)):
        ref = oracle.backward(o0["x"], o["W"], o["A"], o["B"], d[i], o["s"])[1]
        B2 = np.square(o["B"].astype(np.float64))
        least = 2.0 ** -25 if cd == "f16" else 0.0
        off = o["s"] * (np.maximum(u * u * np.abs(d[i]), least) ** 2 @ B2).sum() ** 0.5
        limit = 1e-4 + 4 * off * np.linalg.norm(o0["x"], 2) / np.linalg.norm(ref)
        rel = oracle.rel_l2(to_np(da[i]).astype(np.float64), ref)
        print("dA[%d]: %.2e, bound %.2e" % (i, rel, limit), flush=True)
        assert rel <= limit, "dA[%d]: %.2e > %.2e" % (i, rel, limit)
