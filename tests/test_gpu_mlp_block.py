"""The operators together, as they are used: a block's MLP is trained for two steps (the gated
block, a down projection with drawn dropout, the loss, both backward passes, AdamW), its adapters are
merged, and the merged MLP serves in 8-bit floats."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import dropout as od, fp8 as of, gated as og
from parity import assert_close, oracle_layer, say, to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [5, 200])
def test_train_merge_serve(M):
    say("MLP: train, merge, serve", M)
    D, F, r, p = 256, 512, 16, 0.1
    Ls = [inputs.random_layer(M, F, D, r, seed=1), inputs.random_layer(M, F, D, r, seed=2),
          inputs.random_layer(M, D, F, r, seed=3)]
    gs = [to_gpu(L) for L in Ls]
    qs = [qn.quantize(g["W"], L.block_size, L.double_quant, L.dq_group) for g, L in zip(gs, Ls)]
    x, target = gs[0]["x"], torch.randn(M, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    master = [(g["A"].float(), g["B"].float()) for g in gs]
    state = [[torch.zeros_like(t) for t in ab for _ in (0, 1)] for ab in master]
    A, B = [g["A"].clone() for g in gs], [g["B"].clone() for g in gs]
    seed = torch.tensor([11, 0], dtype=torch.int64).cuda()
    al = [L.alpha for L in Ls]
    for step in (1, 2):
        h, pre, ts = qn.linear_fwd_gated(qs[:2], x, A[:2], B[:2], al[:2], save=True)
        y, t0 = qn.linear_fwd_dropout(qs[2], h, A[2], B[2], al[2], p, seed, save_t=True)
        loss, dy = qn.mse_loss_grad(y, target)
        dh, da2, db2 = qn.linear_bwd_dropout(qs[2], h, dy, A[2], B[2], al[2], p, seed, t_saved=t0)
        dx, das, dbs = qn.linear_bwd_gated(qs[:2], x, dh, A[:2], B[:2], al[:2], pre, t_saved=ts)
        # the step by the oracles, each fed with what the one before handed on
        ops = [oracle_layer(L) for L in Ls]
        for o, a, b in zip(ops, A, B):
            o["A"], o["B"] = to_np(a), to_np(b)
        z = [oracle.forward(to_np(x), o["W"], o["A"], o["B"], o["s"]) for o in ops[:2]]
        assert_close(to_np(h), og.forward(*z, "silu"), "bf16", "h")
        mask, rate = od.drawn_mask(M, F, 11, step - 1, p), od.threshold(p) / 65536
        o = ops[2]
        assert_close(to_np(y), od.forward(to_np(h), o["W"], o["A"], o["B"], o["s"], mask, rate), "bf16", "y")
        rdh, rda, rdb = od.backward(to_np(h), o["W"], o["A"], o["B"], to_np(dy), o["s"], mask, rate)
        assert_close(to_np(dh), rdh, "bf16", "dh")
        assert_close(to_np(da2), rda, "bf16", "dA")
        assert_close(to_np(db2), rdb, "bf16", "dB")
        p64 = to_np(pre).astype(np.float64)
        d = og.backward(p64[:, :F], p64[:, F:], to_np(dh), "silu")
        back = [oracle.backward(to_np(x), o["W"], o["A"], o["B"], d[i], o["s"]) for i, o in enumerate(ops[:2])]
        assert_close(to_np(dx), back[0][0] + back[1][0], "bf16", "dX")
        for i in (0, 1):
            assert_close(to_np(das[i]), back[i][1], "bf16", "dA[%d]" % i)
            assert_close(to_np(dbs[i]), back[i][2], "bf16", "dB[%d]" % i)
        for i, (da, db) in enumerate(zip(das + [da2], dbs + [db2])):
            for j, (m, g, cd) in enumerate(zip(master[i], (da, db), (A[i], B[i]))):
                before = cd.clone()
                qn.adamw_step(m, g, state[i][2 * j], state[i][2 * j + 1], step, 1e-2, param_cd=cd)
                assert torch.isfinite(m).all() and not torch.equal(before, cd)
        seed[1] += 1
    # served: the merged weights in 8-bit floats
    merged = [qn.merge(q, a, b, L.alpha) for q, a, b, L in zip(qs, A, B, Ls)]
    w8 = [qn.quantize_fp8(w) for w in merged]
    gu = [qn.linear_fp8(w, x) for w in w8[:2]]
    for got, w in zip(gu, merged):
        assert_close(to_np(got), of.product(to_np(x), to_np(w))[0], "bf16", "served projection")
    hs = (torch.nn.functional.silu(gu[0].float()) * gu[1].float()).bfloat16()
    ys = qn.linear_fp8(w8[2], hs)
    assert_close(to_np(ys), of.product(to_np(hs), to_np(merged[2]))[0], "bf16", "served output")
    # and it is the trained block: e4m3 rounds each operand by at most 2^-4 (2^-5.8 in the root mean square),
    # which six roundings along the way make 0.045 of the norm
    h = qn.linear_fwd_gated(qs[:2], x, A[:2], B[:2], al[:2])
    y = qn.linear_fwd(qs[2], h, A[2], B[2], al[2])
    assert oracle.rel_l2(to_np(ys).astype(np.float64), to_np(y).astype(np.float64)) <= 0.09
