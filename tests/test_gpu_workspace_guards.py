"""Both passes of the seeded layer and of the gated block in a workspace of just the size that is asked for, between
guards: what lies around it stays, and the results are those of a call with a workspace of its own.  The sizes are those at
which a plan is largest for what the weight holds: a long output of few columns (or few rows), which is decoded in up to
256 tokens (fp32: 128) and whose sums lie in slices, and those on the other side of each rule.

16-bit tolerances are parity.assert_close's: three roundings of half a step of 2^-8 (2^-11) in a row are below 5e-3 of the
norm; fp32: 24 bits of each operand and sums of up to 14336 terms, under 1e-5."""
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import dropout as od
from parity import TORCH_DT, assert_close, say, to_np

pytestmark = pytest.mark.gpu

# tokens, rows, cols, rank, type, block, double quantization with groups of
SHAPES = [(256, 8192, 256, 16, "bf16", 64, 256), (200, 14336, 256, 16, "f16", 32, 0), (256, 10176, 384, 8, "bf16", 64, 256),
          (200, 256, 8192, 16, "bf16", 64, 0), (256, 320, 14272, 8, "f16", 32, 256), (256, 1024, 2048, 64, "bf16", 64, 256),
          (128, 14336, 64, 16, "f32", 64, 0), (127, 192, 5120, 33, "f32", 64, 256), (257, 8192, 128, 16, "bf16", 64, 256),
          (129, 4096, 64, 4, "f32", 32, 0), (17, 9000, 64, 100, "bf16", 64, 100), (60, 100, 77, 8, "bf16", 4, 0)]


def guarded(call, size):
    """The call's tensors in its own workspace and in one of `size` bytes, compared bit by bit."""
    want = call(None)
    ws = torch.full((size + 512,), 77, dtype=torch.uint8).cuda()
    got = call(ws[256:256 + size])
    assert (ws[:256] == 77).all() and (ws[256 + size:] == 77).all()
    flat = lambda v: [t for u in v for t in (flat(u) if isinstance(u, (list, tuple)) else [u]) if t is not None]
    for u, v in zip(flat(got), flat(want)):
        assert torch.equal(u, v)
    return want


@pytest.mark.parametrize("M,N,K,r,cd,block,group", SHAPES)
def test_guards(M, N, K, r, cd, block, group):
    say("workspace guards", M, N, K, r, cd, block, group)
    L = inputs.random_layer(M, N, K, r, seed=M + N, cd=cd, with_dy=True, block_size=block, double_quant=group > 0,
                            dq_group=group or 256)
    ref = oracle.quantize(L.W.numpy(), block, group > 0, group or 256)
    q = qn.quantize(L.W.cuda(), block, group > 0, group or 256)
    dt, drop = TORCH_DT[cd], qn._lib.QLORA_FLAG_DROPOUT
    x, dy, a, b = L.x.cuda(), L.dY.cuda(), L.A.cuda(), L.B.cuda()
    sd, p = torch.tensor([5, 6], dtype=torch.int64).cuda(), 0.25
    fwd, bwd = (qn.workspace_bytes(op, M, N, K, r, dt, drop) for op in (0, 1))
    y, t0 = guarded(lambda ws: qn.linear_fwd_dropout(q, x, a, b, L.alpha, p, sd, save_t=True, workspace=ws), fwd)
    grads = [guarded(lambda ws: qn.linear_bwd_dropout(q, x, dy, a, b, L.alpha, p, sd, workspace=ws, **kw), bwd)
             for kw in (dict(), dict(t_saved=t0), dict(need_dx=False), dict(t_saved=t0, need_dx=False, grad_dtype=dt))]
    W, A, B, xo, dyo = oracle.weight_operand(ref, cd), *(oracle.operand(t, cd) for t in (L.A, L.B, L.x, L.dY))
    mask, rate = od.drawn_mask(M, K, 5, 6, p), od.threshold(p) / 65536
    assert_close(to_np(y), od.forward(xo, W, A, B, L.alpha / r, mask, rate, None), cd, "y")
    for name, g, w in zip(("dX", "dA", "dB"), grads[0], od.backward(xo, W, A, B, dyo, L.alpha / r, mask, rate)):
        assert_close(to_np(g), w, cd, name)

    fwd, bwd = (qn.gated_workspace_bytes(op, (q, q), M, (r, r), dt) for op in (0, 1))
    args = ((q, q), x, [a, a], [b, b], [L.alpha, L.alpha])
    guarded(lambda ws: [qn.linear_fwd_gated(*args, workspace=ws)], fwd)
    h, pre, ts = guarded(lambda ws: qn.linear_fwd_gated(*args, save=True, workspace=ws), fwd)
    for kw in (dict(), dict(t_saved=ts), dict(need_dx=False), dict(t_saved=ts, need_dx=False, grad_dtype=dt)):
        guarded(lambda ws: qn.linear_bwd_gated(args[0], x, dy, *args[2:], pre, workspace=ws, **kw), bwd)


@pytest.mark.parametrize("M,N,K,r,cd,block,group", [(64, 4096, 512, 16, "f32", 64, 0), (1, 1408, 512, 8, "bf16", 64, 256),
                                                    (300, 1088, 1024, 64, "bf16", 64, 256), (129, 320, 77, 9, "f16", 4, 0)])
def test_guards_with_a_stored_mask(M, N, K, r, cd, block, group):
    say("workspace guards, stored mask", M, N, K, r, cd, block, group)
    L = inputs.random_layer(M, N, K, r, seed=M + N, cd=cd, with_dy=True, block_size=block, double_quant=group > 0,
                            dq_group=group or 256)
    q = qn.quantize(L.W.cuda(), block, group > 0, group or 256)
    flags = qn._lib.QLORA_FLAG_DROPOUT | qn._lib.QLORA_FLAG_STORED_MASK
    fwd, bwd = (qn.workspace_bytes(op, M, N, K, r, TORCH_DT[cd], flags) for op in (0, 1))
    args = (L.A.cuda(), L.B.cuda(), L.alpha)
    x, dy = L.x.cuda(), L.dY.cuda()
    mask = (torch.rand(M, K, generator=torch.Generator().manual_seed(1)) < 0.75).to(torch.uint8).cuda()
    drop = dict(dropout_mask=mask, dropout_p=0.25)
    y, t0 = guarded(lambda ws: qn.linear_fwd(q, x, *args, save_t=True, workspace=ws, **drop), fwd)
    for kw in (dict(), dict(t_saved=t0), dict(need_dx=False)):
        guarded(lambda ws: qn.linear_bwd(q, x, dy, *args, workspace=ws, **drop, **kw), bwd)
