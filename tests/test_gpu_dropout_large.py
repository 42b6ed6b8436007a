"""The seeded layer under a path flag on activations past 2^32 bytes, against the rows of calls that stay below.
Each result is within 5e-3 of the exact one (roundings of half a step of 2^-8), two of them within 1e-2 of each other."""
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from bit_nf4_quantized_nibble_amd import inputs
from parity import say
from test_gpu_mlp_layouts import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", ["fused", "dequant"])
def test_activations_past_four_gibibytes(path):
    M, N, K = (1 << 32) // 8192 + 8192 + 3, 64, 4096
    say("seeded dropout: large", path, M, N, K)
    L = inputs.random_layer(8, N, K, 8, seed=3, cd="bf16", with_dy=True)
    q = qn.quantize(L.W.cuda(), L.block_size, L.double_quant, L.dq_group)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    args = (L.A.cuda(), L.B.cuda(), 16.0, 0.25, torch.tensor([1, 2], dtype=torch.int64).cuda())
    y, t0 = qn.linear_fwd_dropout(q, x, *args, save_t=True, path=path)
    dx, da, db = qn.linear_bwd_dropout(q, x, dy, *args, path=path)
    # the mask counts rows: only a call's first rows have the same one, the last have T0 of the whole call alone
    few = 200000
    y2, t2 = qn.linear_fwd_dropout(q, x[:few], *args, save_t=True, path=path)
    dx2, _, _ = qn.linear_bwd_dropout(q, x[:few], dy[:few], *args, t_saved=t2, path=path)
    close(y[:few], y2, "y"), close(t0[:few], t2, "T0"), close(dx[:few], dx2, "dX")
    # T0's mean square of a row is that of x A^T under a mask of 3 in 4: the same far behind as in front
    for part in (t0[few:2 * few], t0[-8192:]):
        assert abs(part.square().mean().item() / t2.square().mean().item() - 1) < 0.1
    # without the last rows' gradients, dA and dB are those of the first
    dy[few:] = 0
    _, da, db = qn.linear_bwd_dropout(q, x, dy, *args, t_saved=t0, need_dx=False, path=path)
    _, da2, db2 = qn.linear_bwd_dropout(q, x[:few], dy[:few], *args, t_saved=t2, need_dx=False, path=path)
    close(da, da2, "dA"), close(db, db2, "dB")
