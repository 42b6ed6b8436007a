"""The gated feed-forward block against the oracle.

Tolerance (parity.assert_close): 5e-3 of the norm for 16-bit types (the operands' roundings: g and u
where they are rounded, the gradients of g and u, dT and T0, each half a step of 2^-8, and the
result's), 1e-5 for fp32."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import gated as og
from parity import TORCH_DT, assert_close, say, to_np

pytestmark = pytest.mark.gpu


def make(M, N, K, rs, cd, seed, bias=False, block=64, dq=True):
    Ls = [inputs.random_layer(M, N, K, r, seed=seed + 13 * i, cd=cd, with_bias=bias, with_dy=True, block_size=block,
                              double_quant=dq) for i, r in enumerate(rs)]
    ops = []
    for L in Ls:
        q = oracle.quantize(L.W.numpy(), L.block_size, L.double_quant, L.dq_group)
        ops.append(dict(W=oracle.weight_operand(q, cd), A=oracle.operand(L.A, cd), B=oracle.operand(L.B, cd),
                        s=L.alpha / L.r, bias=oracle.operand(L.bias, cd) if bias else None))
    g = dict(qs=[qn.quantize(L.W.cuda(), L.block_size, L.double_quant, L.dq_group) for L in Ls], x=Ls[0].x.cuda(),
             a=[L.A.cuda() for L in Ls], b=[L.B.cuda() for L in Ls], al=[L.alpha for L in Ls],
             bias=torch.cat([L.bias for L in Ls]).cuda() if bias else None, dh=Ls[0].dY.cuda())
    return Ls, ops, g


def forward(ops, x):
    return [oracle.forward(x, o["W"], o["A"], o["B"], o["s"], o["bias"]) for o in ops]


CASES = [
    (300, 512, 256, (16, 8), "bf16", "silu", True),       # tiled, a ragged last row tile
    (700, 1280, 512, (8, 8), "f16", "gelu", False),       # tiled, more tiles than one round's cut
    (257, 192, 128, (5, 12), "bf16", "gelu_tanh", True),  # ranks padded to 8, rows not whole tiles
    (65, 64, 64, (64, 1), "f16", "silu", True),
    (520, 1152, 1024, (64, 64), "bf16", "silu", False),
    (100, 200, 256, (8, 4), "bf16", "gelu", True),        # rows not a multiple of 64: by projection
    (90, 128, 128, (8, 8), "f32", "gelu_tanh", False),
    (1, 512, 1024, (16, 16), "bf16", "silu", True),       # decode
    (1, 96, 64, (4, 2), "f32", "gelu", True),
    (33, 256, 1024, (8, 8), "f16", "gelu_tanh", False),
    (130, 320, 320, (96, 8), "bf16", "silu", True),       # a rank the rank-product kernels do not take
    (70, 101, 192, (8, 8), "bf16", "silu", True),         # odd rows
]


@pytest.mark.parametrize("M,N,K,rs,cd,act,bias", CASES)
def test_forward_and_backward(M, N, K, rs, cd, act, bias):
    say("gated", M, N, K, rs, cd, act, bias)
    Ls, ops, g = make(M, N, K, rs, cd, M + N, bias)
    x = oracle.operand(Ls[0].x, cd)
    h, pre, ts = qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], act=act, bias=g["bias"], save=True)
    zg, zu = forward(ops, x)
    assert_close(to_np(h), og.forward(zg, zu, act), cd, "h")
    assert_close(to_np(pre), np.concatenate([zg, zu], 1), cd, "pre")
    for i in range(2):
        assert oracle.rel_l2(to_np(ts[i]).astype(np.float64), x.astype(np.float64) @ ops[i]["A"].astype(np.float64).T) <= 1e-5
    alone = qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], act=act, bias=g["bias"])
    assert torch.equal(alone, h), "saving changes h"

    p64, dh = to_np(pre).astype(np.float64), oracle.operand(Ls[0].dY, cd)
    d = og.backward(p64[:, :N], p64[:, N:], dh, act)
    for gd in (torch.float32, g["x"].dtype):
        dx, das, dbs = qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre, act=act, t_saved=ts,
                                           grad_dtype=gd)
        ref_dx = 0
        for i in range(2):
            o = ops[i]
            rdx, rda, rdb = oracle.backward(x, o["W"], o["A"], o["B"], d[i], o["s"])
            ref_dx = ref_dx + rdx
            assert das[i].dtype == dbs[i].dtype == gd
            assert_close(to_np(das[i]), rda, cd, "dA[%d]" % i)
            assert_close(to_np(dbs[i]), rdb, cd, "dB[%d]" % i)
        assert_close(to_np(dx), ref_dx, cd, "dX")
    none, das2, dbs2 = qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre, act=act, need_dx=False,
                                           grad_dtype=gd)
    assert none is None
    for i in range(2):  # T0 recomputed: the same product
        assert_close(to_np(das2[i]), to_np(das[i]), cd) and assert_close(to_np(dbs2[i]), to_np(dbs[i]), cd)


def test_gradients_are_differences_of_the_loss():
    """f32: directional derivatives of sum(h dh) by central differences of the forward."""
    say("gated: differences")
    Ls, ops, g = make(50, 128, 64, (8, 4), "f32", 5)
    call = lambda x, a, b: (qn.linear_fwd_gated(g["qs"], x, a, b, g["al"], act="gelu_tanh").double() * g["dh"].double()).sum()
    h, pre, ts = qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], act="gelu_tanh", save=True)
    dx, das, dbs = qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre, act="gelu_tanh", t_saved=ts)
    for at, grad in [(("x", None), dx)] + [(("a", i), das[i]) for i in (0, 1)] + [(("b", i), dbs[i]) for i in (0, 1)]:
        v = torch.randn(grad.shape, generator=torch.Generator().manual_seed(1)).cuda()
        v, vals = v / v.norm(), []
        for e in (4e-3, -4e-3):
            t = {"x": g["x"], "a": list(g["a"]), "b": list(g["b"])}
            if at[1] is None:
                t["x"] = g["x"] + e * v
            else:
                t[at[0]][at[1]] = t[at[0]][at[1]] + e * v
            vals.append(call(t["x"], t["a"], t["b"]).item())
        slope, want = (vals[0] - vals[1]) / 8e-3, (grad.double() * v.double()).sum().item()
        # each of the M N terms h dh is off by some 2^-24 sqrt(K) of itself at most, with no direction; the
        # step moves an element by 4e-3 / sqrt(elements), whose square times a third derivative is nothing
        scale = (h.double() * g["dh"].double()).norm().item() * 2.0 ** -24 * 8 / 4e-3
        assert abs(slope - want) <= 4 * scale + 1e-4 * grad.double().norm().item(), at


def test_extreme_values():
    """Saturated activations: the far ends of each, and zeros."""
    say("gated: extremes")
    N, K = 64, 64
    q = qn.quantize(torch.eye(64).cuda(), 64)  # W~ = I exactly: g = u = x
    a, b = torch.zeros(4, K).cuda(), torch.zeros(N, 4).cuda()
    x = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 13.0, -13.0, 40.0, -40.0, 90.0, -90.0, 300.0, -300.0, 1e4, -1e4])
    for cd, big in (("f32", 1e18), ("bf16", 1e18), ("f16", 200.0)):
        dt = TORCH_DT[cd]
        z = torch.zeros(70, K)
        z[:, :16] = x.clamp(-200, 200) if cd == "f16" else x
        z[:, 16], z[:, 17] = big, -big
        z = z.to(dt)
        for act in ("silu", "gelu", "gelu_tanh"):
            args = ((q, q), z.cuda(), [a.to(dt)] * 2, [b.to(dt)] * 2, [1.0, 1.0])
            h, pre, ts = qn.linear_fwd_gated(*args, act=act, save=True)
            zz = to_np(z).astype(np.float64)
            assert np.array_equal(to_np(pre), np.concatenate([to_np(z)] * 2, 1))
            value, slope = og.act(np.clip(zz, -600, 600), act)
            value = np.where(np.abs(zz) > 600, np.maximum(zz, 0), value)
            tol = 4 * torch.finfo(dt).eps
            got = to_np(h).astype(np.float64)
            assert np.allclose(got, value * zz, rtol=tol, atol=1e-6), (cd, act)
            dh = torch.ones(70, N, dtype=dt).cuda()
            dx, _, _ = qn.linear_bwd_gated(args[0], args[1], dh, args[2], args[3], args[4], pre, act=act, t_saved=ts)
            assert np.allclose(to_np(dx).astype(np.float64), zz * slope + value, rtol=tol, atol=1e-2 if cd != "f32" else 1e-5), \
                (cd, act)


def test_streams_graphs_and_refusals():
    say("gated: streams and graphs")
    Ls, ops, g = make(200, 256, 128, (8, 16), "bf16", 3, True)
    f = lambda x: qn.linear_fwd_gated(g["qs"], x, g["a"], g["b"], g["al"], bias=g["bias"], save=True)
    bw = lambda x, pre, ts: qn.linear_bwd_gated(g["qs"], x, g["dh"], g["a"], g["b"], g["al"], pre, t_saved=ts)
    h, pre, ts = f(g["x"])
    grads = bw(g["x"], pre, ts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h2, pre2, ts2 = f(g["x"])
        grads2 = bw(g["x"], pre2, ts2)
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(grads[0], grads2[0]) and torch.equal(grads[1][0], grads2[1][0])
    xs = g["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg, pg, tg = f(xs)
        gg = bw(xs, pg, tg)
    for i in range(3):
        xs.copy_(g["x"] * (1 + i))
        graph.replay()
        torch.cuda.synchronize()
        h3, p3, t3 = f(g["x"] * (1 + i))
        g3 = bw(g["x"] * (1 + i), p3, t3)
        assert torch.equal(hg, h3) and torch.equal(pg, p3) and torch.equal(gg[0], g3[0])
        assert all(torch.equal(u, v) for k in (1, 2) for u, v in zip(gg[k], g3[k]))
    assert f(g["x"][:0])[0].shape == (0, 256)
    x3 = g["x"].view(2, 100, 128)
    assert torch.equal(f(x3)[0], h.view(2, 100, 256))
    bad = [lambda: qn.linear_fwd_gated(g["qs"], g["x"].float(), g["a"], g["b"], g["al"]),
           lambda: qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], act="tanh"),
           lambda: qn.linear_fwd_gated(g["qs"], g["x"], g["a"][::-1], g["b"], g["al"]),
           lambda: qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], bias=g["bias"][:256]),
           lambda: qn.linear_fwd_gated(g["qs"], g["x"], g["a"], g["b"], g["al"], out=h.float()),
           lambda: qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre[:, :256].contiguous()),
           lambda: qn.linear_bwd_gated(g["qs"], g["x"], g["dh"][:7], g["a"], g["b"], g["al"], pre),
           lambda: qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre, t_saved=ts[:1]),
           lambda: qn.linear_bwd_gated(g["qs"], g["x"], g["dh"], g["a"], g["b"], g["al"], pre, grad_dtype=torch.float16)]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
