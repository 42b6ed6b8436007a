"""The layer on activations past 2^32 bytes (x, or dY) against calls on its parts.  Each result is within 5e-3 of the exact one
(roundings of half a step of 2^-8), two of them within 1e-2 of each other."""
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from bit_nf4_quantized_nibble_amd import inputs
from parity import say
from test_gpu_mlp_layouts import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,path", [(64, 4096, "auto"), (64, 4096, "fused"), (4096, 64, "auto"), (4096, 64, "dequant")])
def test_activations_past_four_gibibytes(N, K, path):
    M, part = (1 << 32) // 8192 + 8192 + 3, 200000
    say("layer: large", M, N, K, path)
    L = inputs.random_layer(8, N, K, 8, seed=3, cd="bf16", with_dy=True)
    q = qn.quantize(L.W.cuda(), L.block_size, L.double_quant, L.dq_group)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    args = (L.A.cuda(), L.B.cuda(), 16.0)
    y, t0 = qn.linear_fwd(q, x, *args, save_t=True, path=path)
    dx, da, db = qn.linear_bwd(q, x, dy, *args, t_saved=t0, path=path)
    _, da1, db1 = qn.linear_bwd(q, x, dy, *args, need_dx=False, path=path)
    sums = [0, 0]
    for i in range(0, M, part):
        at = slice(i, min(i + part, M))
        y2, t2 = qn.linear_fwd(q, x[at], *args, save_t=True, path=path)
        dx2, da2, db2 = qn.linear_bwd(q, x[at], dy[at], *args, t_saved=t2, path=path)
        close(y[at], y2, "y"), close(t0[at], t2, "T0"), close(dx[at], dx2, "dX")
        sums = [sums[0] + da2, sums[1] + db2]
    for a, b in ((da, db), (da1, db1)):
        close(a, sums[0], "dA"), close(b, sums[1], "dB")
