"""The operators together, as they are used: an adapter is merged, the merged weight serves as an
8-bit teacher, its top logits train a fresh adapter of the NF4 layer through the distillation loss;
and tokens routed to 8-bit experts give what the experts give one by one."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import distill as od, int8 as oi
from parity import assert_close, oracle_layer, say, to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [7, 200])
def test_merge_serve_distill_train(M):
    say("merge, serve, distill, train", M)
    L = inputs.random_layer(M, 1024, 512, 16, seed=M)
    g = to_gpu(L)
    q = qn.quantize(g["W"], L.block_size, L.double_quant, L.dq_group)
    teacher = qn.quantize_int8(qn.merge(q, g["A"], g["B"] * 20, L.alpha))
    top, index = torch.topk(qn.linear_int8(teacher, g["x"]).float(), 12, dim=1)
    # the student starts from B = 0: its logits are the frozen layer's
    B0 = torch.zeros_like(g["B"])
    logits, t0 = qn.linear_fwd(q, g["x"], g["A"], B0, L.alpha, save_t=True)
    kl = torch.empty(M, device="cuda")
    loss, dlogits = qn.distill_loss_grad(logits, top, index, temperature=2.0, row_kl=kl)
    _, da, db = qn.linear_bwd(q, g["x"], dlogits, g["A"], B0, L.alpha, t_saved=t0, need_dx=False)
    torch.cuda.synchronize()
    # the same chain by the oracles, each fed with what the step before handed on
    mw = to_np(qn.merge(q, g["A"], g["B"] * 20, L.alpha))
    ty, _ = oi.product(to_np(g["x"]), *oi.rows_to_int8(mw))
    assert_close(to_np(qn.linear_int8(teacher, g["x"])), ty, "bf16", "teacher")
    ref, rkl, rdz, _ = od.loss_grad(to_np(logits), to_np(top), to_np(index), 2.0)
    assert abs(loss.item() - ref) <= 1e-5 * max(1.0, ref)
    assert_close(to_np(dlogits), rdz, "bf16", "dlogits")
    o = oracle_layer(L)
    _, rda, rdb = oracle.backward(o["x"], o["W"], o["A"], np.zeros_like(o["B"]), to_np(dlogits).astype(np.float64),
                                  o["s"])
    assert_close(to_np(db), rdb, "bf16", "dB")
    assert not rda.any() and not to_np(da).any()


def test_routed_tokens():
    say("routed tokens")
    E, N, K, M = 8, 384, 256, 150
    gen = torch.Generator().manual_seed(0)
    w = (torch.randn(E, N, K, generator=gen) * 0.05).bfloat16().cuda()
    x = torch.randn(M, K, generator=gen).bfloat16().cuda()
    score = torch.randn(M, E, generator=gen).cuda()
    share, pick = torch.topk(torch.softmax(score, 1), 2, dim=1)
    order = torch.argsort(pick.flatten(), stable=True)
    counts = torch.bincount(pick.flatten(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    q = qn.quantize_int8(w)
    y = qn.linear_int8_experts(q, x[order // 2], offsets)
    out = torch.zeros(M, N, device="cuda")
    out.index_add_(0, order // 2, y.float() * share.flatten()[order][:, None])
    ref = np.zeros((M, N))
    for e in range(E):
        ye, _ = oi.product(to_np(x), *oi.rows_to_int8(to_np(w[e])))
        ref += ye * to_np((share * (pick == e)).sum(1)).astype(np.float64)[:, None]
    assert_close(to_np(out), ref, "bf16", "mixture")
