"""The layer with a drawn dropout mask against the oracle under the mask the generator's definition
gives, and against the call that takes a stored mask."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import dropout as od
from parity import TORCH_DT, assert_close, oracle_layer, say, to_gpu, to_np

pytestmark = pytest.mark.gpu


def seeds(s, o):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v
    return torch.tensor([wrap(s), wrap(o)], dtype=torch.int64).cuda()


def case(M, N, K, r, cd, bias=False, block=64, dq=True, seed=1):
    L = inputs.random_layer(M, N, K, r, seed=seed + M, cd=cd, with_bias=bias, with_dy=True, block_size=block, double_quant=dq)
    g = to_gpu(L)
    return L, g, qn.quantize(g["W"], L.block_size, L.double_quant, L.dq_group)


@pytest.mark.parametrize("M,N,K,r,cd,p,path,bias", [
    (300, 512, 256, 16, "bf16", 0.1, "auto", True),
    (300, 512, 256, 16, "bf16", 0.25, "fused", False),
    (513, 320, 576, 64, "f16", 0.5, "dequant", True),
    (100, 64, 320, 8, "bf16", 0.9, "auto", False),
    (1, 512, 1024, 16, "bf16", 0.1, "auto", True),
    (7, 96, 64, 4, "f32", 0.3, "auto", False),
    (200, 200, 192, 5, "f16", 0.2, "auto", True),       # rank not a multiple of 8, rows not of 64
    (130, 129, 128, 8, "bf16", 0.05, "auto", False),    # odd rows
    (140, 128, 77, 8, "bf16", 0.2, "auto", False),      # cols that end inside a counter's eight
    (90, 64, 77, 8, "f32", 0.2, "auto", True),
    (64, 320, 320, 96, "bf16", 0.1, "auto", False),     # a rank the rank-product kernels do not take
    (2050, 256, 256, 8, "bf16", 0.1, "auto", False),
    (520, 4096, 1024, 64, "bf16", 0.1, "dequant", False),
    (260, 1024, 4096, 64, "bf16", 0.1, "auto", False),  # a cut last round for dX
])
def test_layer(M, N, K, r, cd, p, path, bias):
    say("seeded dropout", M, N, K, r, cd, p, path)
    L, g, q = case(M, N, K, r, cd, bias, dq=N % 128 == 0)
    s, o = 0x9e3779b97f4a7c15, (1 << 63) + 77
    mask = od.drawn_mask(M, K, s, o, p)
    rate = od.threshold(p) / 65536
    sd = seeds(s, o)
    y, t0 = qn.linear_fwd_dropout(q, g["x"], g["A"], g["B"], L.alpha, p, sd, bias=g["bias"], save_t=True, path=path)
    ref = oracle_layer(L)
    assert_close(to_np(y), od.forward(ref["x"], ref["W"], ref["A"], ref["B"], ref["s"], mask, rate, ref["bias"]), cd, "y")
    xm = ref["x"].astype(np.float64) * mask
    assert oracle.rel_l2(to_np(t0).astype(np.float64), xm @ ref["A"].astype(np.float64).T) <= 1e-5
    rdx, rda, rdb = od.backward(ref["x"], ref["W"], ref["A"], ref["B"], ref["dY"], ref["s"], mask, rate)
    for gd in (torch.float32, g["x"].dtype):
        dx, da, db = qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], L.alpha, p, sd, t_saved=t0, path=path,
                                           grad_dtype=gd)
        assert da.dtype == db.dtype == gd
        for name, got, want in (("dX", dx, rdx), ("dA", da, rda), ("dB", db, rdb)):
            assert_close(to_np(got), want, cd, name)
    none, da2, db2 = qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], L.alpha, p, sd, need_dx=False, path=path)
    assert none is None
    assert_close(to_np(da2), rda, cd, "dA, T0 recomputed")
    assert_close(to_np(db2), rdb, cd, "dB, T0 recomputed")


@pytest.mark.parametrize("cd", ["bf16", "f16", "f32"])
def test_the_mask_bit_by_bit(cd):
    """W = 0, B A^T = I: y is x M / (1 - p) itself."""
    say("seeded dropout: the mask", cd)
    for K in (64, 40):
        q = qn.quantize(torch.zeros(64, K).cuda(), 32)
        x = (torch.arange(1, 200 * K + 1) % 13 + 1.0).view(200, K).to(TORCH_DT[cd]).cuda()
        a, b = torch.eye(64, K).to(x.dtype).cuda(), torch.eye(64).to(x.dtype).cuda()
        for s, o in ((0, 0), (1, 0), (0, 1), (1 << 63, (1 << 64) - 1), (0xffffffff, 1 << 32)):
            y = qn.linear_fwd_dropout(q, x, a, b, 64.0, 0.5, seeds(s, o))
            want = x.float().cpu().numpy() * od.drawn_mask(200, K, s, o, 0.5) * 2
            assert np.array_equal(to_np(y)[:, :K].astype(np.float32), want)


@pytest.mark.parametrize("p", [0.0, 0.25, 0.97])
def test_rates_and_the_stored_mask(p):
    say("seeded dropout: against the stored mask", p)
    L, g, q = case(150, 192, 128, 8, "bf16")
    sd = seeds(5, 6)
    rate = od.threshold(p) / 65536
    mask = torch.from_numpy(od.drawn_mask(150, 128, 5, 6, p)).cuda()
    y = qn.linear_fwd_dropout(q, g["x"], g["A"], g["B"], L.alpha, p, sd)
    assert_close(to_np(y), to_np(qn.linear_fwd(q, g["x"], g["A"], g["B"], L.alpha, dropout_mask=mask, dropout_p=rate)),
                 "bf16")
    if p == 0.0:
        assert_close(to_np(y), to_np(qn.linear_fwd(q, g["x"], g["A"], g["B"], L.alpha)), "bf16")
    dx, da, db = qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], L.alpha, p, sd)
    rx, ra, rb = qn.linear_bwd(q, g["x"], g["dY"], g["A"], g["B"], L.alpha, dropout_mask=mask, dropout_p=rate)
    assert_close(to_np(da), to_np(ra), "bf16") and assert_close(to_np(db), to_np(rb), "bf16")
    assert_close(to_np(dx), to_np(rx), "bf16")


def test_a_captured_call_draws_anew():
    say("seeded dropout: graphs")
    L, g, q = case(300, 256, 256, 16, "bf16")
    sd = seeds(3, 0)

    def step():
        y, t0 = qn.linear_fwd_dropout(q, g["x"], g["A"], g["B"], L.alpha, 0.3, sd, save_t=True)
        return (y, t0) + qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], L.alpha, 0.3, sd, t_saved=t0)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        sd[1:].add_(1)  # the program's own count
    seen = []
    for i in range(4):
        sd[1] = 10 + i
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert sd[1].item() == 11 + i
        sd[1] = 10 + i
        assert all(torch.equal(u, v) for u, v in zip(got, step()))
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])
    side = torch.cuda.Stream()
    sd[1] = 10
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    side.synchronize()
    assert torch.equal(again[0], seen[0])


def test_refusals_and_shapes():
    say("seeded dropout: refusals")
    L, g, q = case(20, 64, 64, 8, "bf16")
    sd = seeds(1, 2)
    ok = (q, g["x"], g["A"], g["B"], L.alpha)
    x3 = g["x"].view(4, 5, 64)
    assert torch.equal(qn.linear_fwd_dropout(q, x3, *ok[2:], 0.1, sd), qn.linear_fwd_dropout(*ok, 0.1, sd).view(4, 5, 64))
    assert qn.linear_fwd_dropout(q, g["x"][:0], *ok[2:], 0.1, sd).shape == (0, 64)
    for bad in (lambda: qn.linear_fwd_dropout(*ok, 1.0, sd), lambda: qn.linear_fwd_dropout(*ok, -0.5, sd),
                lambda: qn.linear_fwd_dropout(*ok, 0.1, sd.cpu()), lambda: qn.linear_fwd_dropout(*ok, 0.1, sd.int()),
                lambda: qn.linear_fwd_dropout(*ok, 0.1, sd[:1]), lambda: qn.linear_fwd_dropout(*ok, 0.1, sd, path="other"),
                lambda: qn.linear_fwd_dropout(q, g["x"], g["A"][:, :32].contiguous(), g["B"], 1.0, 0.1, sd),
                lambda: qn.linear_bwd_dropout(q, g["x"], g["dY"][:3], g["A"], g["B"], 1.0, 0.1, sd),
                lambda: qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], 1.0, 0.1, sd, grad_dtype=torch.float16),
                lambda: qn.linear_bwd_dropout(q, g["x"], g["dY"], g["A"], g["B"], 1.0, 0.1, sd, t_saved=g["x"].float())):
        with pytest.raises((ValueError, TypeError)):
            bad()
