"""The gated block and the layer with a drawn mask in layouts and sizes away from the tuned kernels':
blocks that run across rows, block sizes that are no power of two or shorter than eight, columns
that end inside a stage, ranks past 64, each side of the sizes at which a call goes another way.

Tolerances are parity.assert_close's.  16-bit: an operand, an intermediate (g, u, dg, du) and the
result are each rounded by at most half a step of 2^-8 (2^-11), three such roundings in a row are
off by 3 * 2^-9 / sqrt(3) of the norm or less, under 5e-3.  fp32: operands are kept to 24 bits in
three parts of 8, the products left out are below 2^-22 of the largest, sums of up to a few thousand
terms in fp32 add some 2^-24 sqrt(K): under 1e-5."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
import oracle
from bit_nf4_quantized_nibble_amd import inputs
from oracle import dropout as od
from oracle import gated as og
from parity import TORCH_DT, assert_close, say, to_np

pytestmark = pytest.mark.gpu

# tokens, rows, cols, rank, type, block, double quantization with groups of
LAYOUTS = [
    (1, 64, 65, 1, "bf16", 2, 0),            # eight weights in up to five blocks
    (3, 128, 63, 7, "f16", 4, 256),
    (70, 60, 77, 5, "f32", 6, 0),            # no power of two
    (129, 96, 130, 80, "bf16", 96, 100),     # a rank past 64, groups that are no power of two
    (33, 37, 192, 33, "bf16", 64, 256),      # odd rows
    (40, 50, 64, 200, "f32", 32, 0),         # a rank of four stages
    (128, 320, 256, 8, "f16", 64, 256),      # the last size whose weight is decoded in the product (fp32)
    (129, 320, 256, 8, "f32", 64, 0),
    (128, 192, 320, 24, "f32", 32, 256),
    (256, 129, 256, 16, "bf16", 64, 256),    # and in 16 bits
    (257, 129, 256, 16, "bf16", 64, 0),
    (1, 1, 64, 1, "f32", 64, 0),             # one row, one token
    (600, 2112, 100, 12, "bf16", 64, 0),     # enough tiles that none is cut
    (2048, 1856, 70, 70, "f16", 64, 256),    # the larger tiles
    (2050, 64, 1030, 16, "bf16", 64, 0),
    (1030, 192, 1100, 9, "f32", 64, 256),
    (300, 1024, 1088, 16, "bf16", 64, 256),  # about where the tuned kernels take over
    (1030, 2048, 2112, 8, "bf16", 64, 256),
]


def layer(M, N, K, r, cd, block, group, seed, bias=False):
    L = inputs.random_layer(M, N, K, r, seed=seed, cd=cd, with_bias=bias, with_dy=True, block_size=block,
                            double_quant=group > 0, dq_group=group or 256)
    q = oracle.quantize(L.W.numpy(), block, group > 0, group or 256)
    o = dict(W=oracle.weight_operand(q, cd), A=oracle.operand(L.A, cd), B=oracle.operand(L.B, cd), s=L.alpha / L.r,
             x=oracle.operand(L.x, cd), dY=oracle.operand(L.dY, cd), bias=oracle.operand(L.bias, cd) if bias else None)
    return L, o, qn.quantize(L.W.cuda(), block, group > 0, group or 256)


@pytest.mark.parametrize("M,N,K,r,cd,block,group", LAYOUTS)
def test_gated(M, N, K, r, cd, block, group):
    say("gated layouts", M, N, K, r, cd, block, group)
    bias, act = M % 2 == 0, ("silu", "gelu", "gelu_tanh")[M % 3]
    r2 = max(1, r // 2)
    (L0, o0, q0), (L1, o1, q1) = layer(M, N, K, r, cd, block, group, M, bias), layer(M, N, K, r2, cd, block, group, M + 1, bias)
    x, dh = L0.x.cuda(), L0.dY.cuda()
    args = ((q0, q1), x, [L0.A.cuda(), L1.A.cuda()], [L0.B.cuda(), L1.B.cuda()], [L0.alpha, L1.alpha])
    b = torch.cat([L0.bias, L1.bias]).cuda() if bias else None
    h, pre, ts = qn.linear_fwd_gated(*args, act=act, bias=b, save=True)
    z = [oracle.forward(o0["x"], o["W"], o["A"], o["B"], o["s"], o["bias"]) for o in (o0, o1)]
    assert_close(to_np(h), og.forward(z[0], z[1], act), cd, "h")
    assert_close(to_np(pre), np.concatenate(z, 1), cd, "pre")
    for t, o in zip(ts, (o0, o1)):
        assert oracle.rel_l2(to_np(t).astype(np.float64), o0["x"].astype(np.float64) @ o["A"].astype(np.float64).T) <= 1e-5
    assert torch.equal(qn.linear_fwd_gated(*args, act=act, bias=b), h)

    p64 = to_np(pre).astype(np.float64)
    d = og.backward(p64[:, :N], p64[:, N:], o0["dY"], act)
    ref = [oracle.backward(o0["x"], o["W"], o["A"], o["B"], d[i], o["s"]) for i, o in enumerate((o0, o1))]
    # dA = dT^T x, dT = s d B: d is rounded to the type, each element by u = eps / 2 of itself at most and so by
    # u / sqrt(3) in the mean square, independently; dT is then off by s u / sqrt(3) sqrt(sum_n d^2 B^2), however much
    # its sum cancels, and with one token and rank 1 every element of dA by the same factor.  Four times that
    # lies beside the 5e-3 of the other roundings (the first run, without it, had 1.3e-2 at M = r = 1).
    u = 0.0 if cd == "f32" else torch.finfo(TORCH_DT[cd]).eps / 2
    limit = [(1e-5 if cd == "f32" else 5e-3) + 4 * u / 3 ** 0.5 * o["s"]
             * (np.square(d[i]) @ np.square(o["B"].astype(np.float64))).sum() ** 0.5
             * np.linalg.norm(o0["x"], 2) / np.linalg.norm(ref[i][1]) for i, o in enumerate((o0, o1))]
    back = lambda **kw: qn.linear_bwd_gated(args[0], x, dh, *args[2:], pre, act=act, **kw)
    for kw in (dict(t_saved=ts), dict(grad_dtype=x.dtype), dict(t_saved=ts, need_dx=False), dict(need_dx=False)):
        dx, da, db = back(**kw)
        for i in range(2):
            assert oracle.rel_l2(to_np(da[i]).astype(np.float64), ref[i][1]) <= limit[i], "dA[%d]" % i
            assert_close(to_np(db[i]), ref[i][2], cd, "dB[%d]" % i)
        if kw.get("need_dx", True):
            assert_close(to_np(dx), ref[0][0] + ref[1][0], cd, "dX")
        else:
            assert dx is None
    again = back(t_saved=ts)
    assert torch.equal(again[0], back(t_saved=ts)[0]) and torch.equal(again[1][0], back(t_saved=ts)[1][0])


@pytest.mark.parametrize("M,N,K,r,cd,block,group", LAYOUTS)
def test_dropout(M, N, K, r, cd, block, group):
    say("seeded dropout layouts", M, N, K, r, cd, block, group)
    p, s, o = 0.25, 12345678901234567, 1 << 40
    L, ref, q = layer(M, N, K, r, cd, block, group, M, M % 2 == 1)
    mask, rate = od.drawn_mask(M, K, s, o, p), od.threshold(p) / 65536
    sd = torch.tensor([s, o], dtype=torch.int64).cuda()
    x, dy, a, b = L.x.cuda(), L.dY.cuda(), L.A.cuda(), L.B.cuda()
    y, t0 = qn.linear_fwd_dropout(q, x, a, b, L.alpha, p, sd, bias=None if L.bias is None else L.bias.cuda(), save_t=True)
    assert_close(to_np(y), od.forward(ref["x"], ref["W"], ref["A"], ref["B"], ref["s"], mask, rate, ref["bias"]), cd, "y")
    xm = ref["x"].astype(np.float64) * mask
    assert oracle.rel_l2(to_np(t0).astype(np.float64), xm @ ref["A"].astype(np.float64).T) <= 1e-5
    want = od.backward(ref["x"], ref["W"], ref["A"], ref["B"], ref["dY"], ref["s"], mask, rate)
    back = lambda **kw: qn.linear_bwd_dropout(q, x, dy, a, b, L.alpha, p, sd, **kw)
    for kw in (dict(t_saved=t0), dict(grad_dtype=x.dtype), dict(t_saved=t0, need_dx=False), dict(need_dx=False)):
        got = back(**kw)
        for name, g, w in zip(("dX", "dA", "dB"), got, want):
            if g is not None:
                assert_close(to_np(g), w, cd, name)
        assert (got[0] is None) == (not kw.get("need_dx", True))
    assert all(torch.equal(u, v) for u, v in zip(back(), back()))


@pytest.mark.parametrize("M,N,K,cd", [(20, 96, 80, "bf16"), (20, 96, 80, "f32"), (20, 128, 128, "f32"), (20, 130, 128, "f16"),
                                      (300, 96, 80, "bf16"), (300, 1088, 1024, "bf16"), (700, 2112, 2048, "bf16")])
def test_a_row_that_is_no_number_stays_alone(M, N, K, cd):
    """x, dh and dY of one row infinite or NaN: every other row is what it was."""
    say("layouts: infinities", M, N, K, cd)
    L, o, q = layer(M, N, K, 8, cd, 32, 256, 3)
    dt = TORCH_DT[cd]
    a, b = L.A.cuda(), L.B.cuda()
    sd = torch.tensor([1, 2], dtype=torch.int64).cuda()
    rest = torch.arange(M) != M - 1
    run = lambda x, dh, pre: (qn.linear_fwd_gated((q, q), x, [a, a], [b, b], [8.0, 8.0], save=True)[:2]
                              + (qn.linear_fwd_dropout(q, x, a, b, 8.0, 0.3, sd),
                                 qn.linear_bwd_gated((q, q), L.x.cuda(), dh, [a, a], [b, b], [8.0, 8.0], pre)[0],
                                 qn.linear_bwd_dropout(q, L.x.cuda(), dh, a, b, 8.0, 0.3, sd)[0]))
    pre = qn.linear_fwd_gated((q, q), L.x.cuda(), [a, a], [b, b], [8.0, 8.0], save=True)[1]
    clean = run(L.x.cuda(), L.dY.cuda(), pre)
    for bad in (float("inf"), float("nan")):
        x, dh = L.x.cuda(), L.dY.cuda()
        x[M - 1, K - 1] = bad
        dh[M - 1, N - 1] = bad
        for got, want in zip(run(x, dh, pre), clean):
            assert torch.equal(got[rest], want[rest]) and not torch.isfinite(got[M - 1].float()).all()


@pytest.mark.parametrize("M,N,K,cd", [(60, 100, 77, "bf16"), (60, 128, 128, "f32"), (300, 100, 128, "f16"), (300, 2112, 2048, "bf16")])
def test_nothing_behind_the_outputs(M, N, K, cd):
    """Outputs inside larger buffers, a workspace of just the size asked for: what lies around them stays."""
    say("layouts: guards", M, N, K, cd)
    L, o, q = layer(M, N, K, 8, cd, 4 if K % 32 else 32, 0, 5)
    dt = TORCH_DT[cd]
    args = (L.x.cuda(), L.A.cuda(), L.B.cuda())
    sd = torch.tensor([1, 2], dtype=torch.int64).cuda()
    need = (qn.gated_workspace_bytes(qn._lib.QLORA_OP_FWD, (q, q), M, (8, 8), dt),
            qn.workspace_bytes(qn._lib.QLORA_OP_FWD, M, N, K, 8, dt, qn._lib.QLORA_FLAG_DROPOUT))
    calls = (lambda out, ws: qn.linear_fwd_gated((q, q), args[0], [args[1]] * 2, [args[2]] * 2, [8.0, 8.0], out=out, workspace=ws),
             lambda out, ws: qn.linear_fwd_dropout(q, *args, 8.0, 0.3, sd, out=out, workspace=ws))
    for call, n in zip(calls, need):
        want = call(None, None)
        room, ws = torch.full((M * N + 512,), 7.0, dtype=dt).cuda(), torch.full((n + 512,), 77, dtype=torch.uint8).cuda()
        got = call(room[256:256 + M * N].view(M, N), ws[256:256 + n])
        assert torch.equal(got, want)
        assert (room[:256] == 7).all() and (room[256 + M * N:] == 7).all()
        assert (ws[:256] == 77).all() and (ws[256 + n:] == 77).all()
        with pytest.raises(ValueError):
            call(None, ws[:n - 1])


@pytest.mark.parametrize("M,N,K,cd", [(100, 96, 80, "bf16"), (100, 128, 128, "f32"), (400, 1088, 1024, "bf16"), (700, 2112, 2048, "f16")])
def test_two_graphs_and_two_streams(M, N, K, cd):
    """Both blocks of a layer captured in two graphs that share a workspace, replayed with eager calls between."""
    say("layouts: graphs", M, N, K, cd)
    L, o, q = layer(M, N, K, 8, cd, 32, 256, 7)
    x0, dy, a, b = L.x.cuda(), L.dY.cuda(), L.A.cuda(), L.B.cuda()
    sd = torch.tensor([3, 0], dtype=torch.int64).cuda()
    dt = TORCH_DT[cd]
    size = max([qn.gated_workspace_bytes(op, (q, q), M, (8, 8), dt) for op in (0, 1)]
               + [qn.workspace_bytes(op, M, N, K, 8, dt, qn._lib.QLORA_FLAG_DROPOUT) for op in (0, 1)])
    ws = torch.empty(size, dtype=torch.uint8).cuda()

    def gated(x, w=None):
        h, pre, ts = qn.linear_fwd_gated((q, q), x, [a, a], [b, b], [8.0, 8.0], save=True, workspace=w)
        dx, da, db = qn.linear_bwd_gated((q, q), x, dy, [a, a], [b, b], [8.0, 8.0], pre, t_saved=ts, workspace=w)
        return [h, pre, dx] + ts + da + db

    def drop(x, w=None):
        y, t0 = qn.linear_fwd_dropout(q, x, a, b, 8.0, 0.3, sd, save_t=True, workspace=w)
        return [y, t0] + list(qn.linear_bwd_dropout(q, x, dy, a, b, 8.0, 0.3, sd, t_saved=t0, workspace=w))

    xs = x0.clone()
    graphs, outs = [], []
    for f in (gated, drop):
        f(xs, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f(xs, ws))
        graphs.append(graph)
    for i in range(3):
        xs.copy_(x0 * (1 + i))
        sd[1] = i
        for graph, out, f in zip(graphs, outs, (gated, drop)):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(out, f(x0 * (1 + i))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    here = gated(x0)
    with torch.cuda.stream(side):  # at the same time
        there = drop(x0)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(here, gated(x0)))
    assert all(torch.equal(u, v) for u, v in zip(there, drop(x0)))


@pytest.mark.parametrize("M,N,K,cd", [(50, 96, 80, "bf16"), (700, 2112, 2048, "bf16")])
def test_a_saved_product_of_one_projection_only(M, N, K, cd):
    """The C call with T0 of the gate alone: both are formed again."""
    say("layouts: one T0", M, N, K, cd)
    L, o, q = layer(M, N, K, 8, cd, 32, 256, 11)
    x, dy, a, b = L.x.cuda(), L.dY.cuda(), [L.A.cuda()] * 2, [L.B.cuda()] * 2
    h, pre, ts = qn.linear_fwd_gated((q, q), x, a, b, [8.0, 8.0], save=True)
    want = qn.linear_bwd_gated((q, q), x, dy, a, b, [8.0, 8.0], pre)
    ga = qn._GatedArgs((q, q), [8, 8], a, b, [8.0, 8.0])
    new = lambda *shape: torch.empty(*shape, dtype=torch.float32).cuda()
    dx, da, db = torch.empty_like(x), [new(8, K), new(8, K)], [new(N, 8), new(N, 8)]
    ws = torch.empty(qn.gated_workspace_bytes(qn._lib.QLORA_OP_BWD, (q, q), M, (8, 8), x.dtype), dtype=torch.uint8).cuda()
    for t in ((ts[0].data_ptr(), None), (None, ts[1].data_ptr())):
        qn._launch(x.device, qn._lib.lib().qlora_linear_bwd_gated, ga.w, x.data_ptr(), dy.data_ptr(), pre.data_ptr(), M, ga.a, ga.b,
                   ga.r, ga.alpha, 0, 0, qn.dtype_code(x.dtype), qn._Two(*t), 0, dx.data_ptr(), qn._two(da), qn._two(db),
                   ws.data_ptr(), ws.numel())
        assert torch.equal(dx, want[0]) and all(torch.equal(u, v) for u, v in zip(da + db, want[1] + want[2]))


def close(got, want, what):
    """Two results of different kernels, each within 5e-3 of the exact one, on the GPU in row blocks."""
    num = den = 0.0
    for u, v in zip(got.split(1 << 14), want.split(1 << 14)):
        num += (u.double() - v.double()).square().sum().item()
        den += v.double().square().sum().item()
    assert num ** 0.5 <= 1e-2 * den ** 0.5, (what, (num / den) ** 0.5)


def test_activations_past_two_gibibytes():
    """Offsets past 2^31 bytes in pre, dg and du (gated) and in x (dropout): the call against its two halves."""
    M, N, K = 270336, 2048, 128
    say("layouts: large", M, N, K)
    L, o, q = layer(8, N, K, 8, "bf16", 64, 256, 13)
    gen = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    x, dh, a, b = draw(M, K), draw(M, N), [L.A.cuda()] * 2, [L.B.cuda()] * 2
    f = lambda x: qn.linear_fwd_gated((q, q), x, a, b, [16.0, 16.0], save=True)
    g = lambda x, dh, pre, ts: qn.linear_bwd_gated((q, q), x, dh, a, b, [16.0, 16.0], pre, t_saved=ts)
    half = M // 2
    h, pre, ts = f(x)
    dx, da, db = g(x, dh, pre, ts)
    sums = [0, 0]
    for i in (slice(0, half), slice(half, M)):
        h2, pre2, ts2 = f(x[i])
        dx2, da2, db2 = g(x[i], dh[i], pre2, ts2)
        close(h[i], h2, "h"), close(pre[i], pre2, "pre"), close(dx[i], dx2, "dX")
        sums = [sums[0] + da2[0], sums[1] + db2[1]]
    close(da[0], sums[0], "dA"), close(db[1], sums[1], "dB")
    del h, pre, ts, dx, h2, pre2, ts2, dx2, dh

    M, N, K = 266240, 64, 4096  # the mask counts rows, so the second half has another one: rows are compared
    L, o, q = layer(8, N, K, 8, "bf16", 64, 256, 14)
    x, dy, sd = draw(M, K), draw(M, N), torch.tensor([1, 2], dtype=torch.int64).cuda()
    args = (L.A.cuda(), L.B.cuda(), 16.0, 0.25, sd)
    y, t0 = qn.linear_fwd_dropout(q, x, *args, save_t=True)
    dx, da, db = qn.linear_bwd_dropout(q, x, dy, *args, t_saved=t0)
    x[half:] = 0
    dy[half:] = 0
    y2, t2 = qn.linear_fwd_dropout(q, x[:half], *args, save_t=True)
    dx2, da2, db2 = qn.linear_bwd_dropout(q, x[:half], dy[:half], *args, t_saved=t2)
    close(y[:half], y2, "y"), close(t0[:half], t2, "T0"), close(dx[:half], dx2, "dX")
    y, t0 = qn.linear_fwd_dropout(q, x, *args, save_t=True)
    dx, da, db = qn.linear_bwd_dropout(q, x, dy, *args, t_saved=t0)
    close(da, da2, "dA"), close(db, db2, "dB")
    assert not y[half:].any() and not dx[half:].any()
