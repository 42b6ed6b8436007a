"""The distillation loss and its gradient against the oracle.

Tolerances, from the arithmetic (u = 2^-24): an exponent (z - max) / T carries at most 4 u of its
own size A (difference, 1 / T, product, the change of base), its exponential 4 u more; a sum over
the vocabulary in fp32 adds at most u for each term of one thread's chain (at most V / 256 terms)
and of the trees (at most 32); so a probability is off by at most
  rel = u (8 A + V / 256 + 64)
of itself.  The gradient at an entry is off by |w| T (q + p) rel, then rounded once into its type
(half a step); kl by rel times the size of the numbers that cancel in it (the oracle's kl_mag)."""
import warnings

import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from oracle import distill as od
from parity import TORCH_DT, say, to_np

pytestmark = pytest.mark.gpu


def make(n, V, k, cd, seed, spread=3.0, pad=0, td="f32"):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(n, V, generator=g) * spread
    z = (t + 0.5 * torch.randn(n, V, generator=g)).to(TORCH_DT[cd])
    kk = min(k, V)
    u, idx = torch.topk(t, kk, dim=1)
    if kk < k:  # more slots than vocabulary entries: the rest are absent
        u = torch.cat([u, torch.zeros(n, k - kk)], 1)
        idx = torch.cat([idx, torch.full((n, k - kk), -1)], 1)
    if pad:
        buf = torch.full((n, V + pad), float("nan"), dtype=TORCH_DT[cd])
        buf[:, :V] = z
        z = buf[:, :V]
    return z, u.to(TORCH_DT[td]), idx


def bounds(z, u, T, V):
    zf = np.where(np.isfinite(to_np(z)), to_np(z), np.nan).astype(np.float64)
    uf = np.where(np.isfinite(to_np(u)), to_np(u), np.nan).astype(np.float64)
    with np.errstate(all="ignore"), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # rows without a finite value
        A = np.nanmax(np.nanmax(zf, 1) - np.nanmin(zf, 1)) / T
        B = np.nanmax(np.nanmax(uf, 1) - np.nanmin(uf, 1)) / T
    # exponentials of less than -110 vanish in fp32 and in the bound's absolute term
    A = min(max(np.nan_to_num(A), np.nan_to_num(B)), 110.0)
    return 2.0 ** -24 * (8 * A + V / 256 + 64)


def check(z, u, idx, T=1.0, w=None, grad=True, in_place=False, bits=64, dz_pad=None):
    n, V = z.shape
    cd = z.dtype
    dev = lambda t: None if t is None else t.cuda()
    zc = dev(z)
    if z.stride(0) != V and n > 1:  # keep the row stride on the GPU
        buf = torch.full((n, z.stride(0)), float("nan"), dtype=cd, device="cuda")
        buf[:, :V] = zc
        zc = buf[:, :V]
    before = zc.clone()
    ix = idx.to(torch.int32 if bits == 32 else torch.int64)
    dl = None
    if in_place:
        dl = zc
    elif dz_pad is not None:
        frame = torch.full((n, V + dz_pad), 7.0, dtype=cd, device="cuda")
        dl = frame[:, :V]
    kl = torch.full((n,), -1.0, device="cuda")
    loss, dz = qn.distill_loss_grad(zc, dev(u), dev(ix), temperature=T, weight=dev(w), need_grad=grad, dlogits=dl,
                                    row_kl=kl)
    torch.cuda.synchronize()
    ref_loss, ref_kl, ref_dz, mag = od.loss_grad(to_np(z), to_np(u), to_np(idx), T, None if w is None else to_np(w))
    rel = bounds(z, u, T, V)
    wn = np.full(n, 1.0 / n) if w is None else to_np(w).astype(np.float64)
    live = wn != 0
    tol_kl = 1.1 * rel * mag + 1e-37
    got = to_np(kl).astype(np.float64)
    same = (got == ref_kl) | (np.isnan(got) & np.isnan(ref_kl))
    assert np.all(same | (np.abs(got - ref_kl) <= tol_kl)), (got, ref_kl)
    tol = float((np.abs(wn[live]) * (tol_kl[live] + 2.0 ** -22 * np.abs(np.nan_to_num(ref_kl[live], posinf=0)))).sum())
    g0 = float(loss.item())
    assert g0 == ref_loss or (np.isnan(g0) and np.isnan(ref_loss)) or abs(g0 - ref_loss) <= tol + 1e-37, (g0, ref_loss)
    if not grad:
        assert dz is None and torch.equal(zc.nan_to_num(7.5), before.nan_to_num(7.5))
        return loss, dz
    p_plus_q = np.abs(ref_dz) + 2 * shares(u, idx, T, V, n) * (np.abs(wn) * T)[:, None]
    tol = 1.1 * (rel * p_plus_q + torch.finfo(cd).eps / 2 * np.abs(ref_dz))
    tol += (np.abs(wn) * T)[:, None] * 2.0 ** -120 + float(torch.finfo(cd).tiny) * torch.finfo(cd).eps / 2
    got = to_np(dz).astype(np.float64)
    bad = ~((np.abs(got - ref_dz) <= tol) | (np.isnan(got) & np.isnan(ref_dz)))
    assert not bad.any(), "%d of %d beyond the bound, first at %s: %r, expected %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref_dz[bad][0])
    dead = ~live | ~np.any((to_np(idx) >= 0) & (to_np(idx) < V) & (to_np(u) != -np.inf), axis=1)
    assert not got[dead].any()
    if dz_pad:
        assert torch.equal(frame[:, V:], torch.full((n, dz_pad), 7.0, dtype=cd, device="cuda")), "padding written"
    if not in_place:
        assert torch.equal(zc.nan_to_num(7.5), before.nan_to_num(7.5)), "logits changed"
    return loss, dz


def shares(u, idx, T, V, n):
    """The teacher's distribution scattered over the vocabulary (for the bound)."""
    out = np.zeros((n, V))
    un, ix = to_np(u).astype(np.float64) / T, to_np(idx)
    for i in range(n):
        here = (ix[i] >= 0) & (ix[i] < V) & (un[i] != -np.inf)
        if here.any():
            e = np.exp(np.nan_to_num(un[i][here] - un[i][here].max()))
            np.add.at(out[i], ix[i][here], e / e.sum())
    return out


CASES = [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 64, 8), (4, 1000, 16), (3, 4097, 33), (9, 8192, 64), (2, 32000, 100),
         (3, 50257, 5), (2, 65536, 256), (2, 100003, 1024), (2, 131072, 7), (3, 128000, 64), (2, 151936, 20),
         (2, 163840, 9), (2, 200001, 50), (300, 513, 12)]


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V,k", CASES)
def test_loss_and_gradient(n, V, k, cd):
    say("distill", n, V, k, cd)
    z, u, idx = make(n, V, k, cd, n + V + k)
    check(z, u, idx, T=1.0, bits=32 if V % 2 else 64)


# Up to 256 long rows are cut into parts; others stay whole, in registers or (the longest) read twice.
WHOLE = [(2100, 1, 1), (2100, 100, 128), (2101, 4099, 40), (2100, 300, 129), (65, 8200, 16), (257, 9001, 200), (300, 16391, 20), (300, 32760, 128), (270, 20000, 130), (70, 32768, 30), (66, 65536, 64), (65, 128000, 33),
         (65, 150001, 12), (65, 170007, 5),
         (258, 40000, 30), (257, 65001, 140), (180, 150001, 12), (180, 170007, 5), (256, 262145, 9), (96, 131072, 17)]


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V,k", WHOLE)
def test_whole_rows(n, V, k, cd):
    say("whole rows", n, V, k, cd)
    z, u, idx = make(n, V, k, cd, n + V + k)
    w = torch.rand(n, generator=torch.Generator().manual_seed(1)) / n
    w[torch.randperm(n, generator=torch.Generator().manual_seed(2))[: n // 3]] = 0
    idx[n - 1] = -1                       # rows left out next to each other and at the end
    idx[5:8] = -1
    idx[9, : k // 2] = idx[9, k // 2]
    check(z, u, idx, T=0.9, w=w, in_place=n % 2 == 0)
    check(z, u, idx, T=0.9, w=w, grad=False)


@pytest.mark.parametrize("V", [8300, 40000, 120001, 171000])
@pytest.mark.parametrize("n", [64, 65, 257])
def test_special_values_in_long_rows(V, n):
    """The same rows with few of them (cut into parts) and with more (whole)."""
    say("special values", n, V)
    z, u, idx = make(n, V, 8, "bf16", V)
    lowest = torch.finfo(z.dtype).min
    z[0, :] = float("-inf")                       # nothing allowed: NaN
    z[1, V - 1] = float("nan")
    z[2, V // 2] = float("inf")
    z[3, : V - 9] = float("-inf")                 # whole stretches of nothing
    z[4, 100:] = float("-inf")
    z[5, :] = lowest                              # uniform
    z[6, :] = lowest
    z[6, V - 1] = 3.0
    z[7, idx[7, 2]] = float("-inf")               # the teacher wants a forbidden entry
    idx[3] = torch.arange(V - 8, V)
    idx[4] = torch.arange(0, 8)
    idx[5] = torch.arange(V - 8, V)
    idx[6] = V - 1
    kl = torch.empty(n, device="cuda")
    loss, dz = qn.distill_loss_grad(z.cuda(), u.cuda(), idx.cuda(), row_kl=kl)
    kl, dz = to_np(kl), to_np(dz)
    assert np.isnan(kl[:3]).all() and np.isnan(dz[:3]).all() and kl[7] == np.inf and np.isfinite(dz[7]).all()
    assert np.isnan(loss.item()) and np.isfinite(kl[8:]).all()
    keep = [3, 4, 5, 6] + list(range(8, 20))
    w = torch.zeros(n)
    w[keep] = 0.25
    check(z, u, idx, w=w)
    check(z, u, idx, w=w, grad=False)
    check(z, u, idx, w=w, in_place=True)


@pytest.mark.parametrize("T", [0.05, 0.7, 2.0, 50.0])
@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V", [(6, 3001), (6, 40009), (65, 20000)])
def test_temperatures(n, V, T, cd):
    say("temperature", n, V, T, cd)
    check(*make(n, V, 24, cd, 5), T=T)


@pytest.mark.parametrize("td", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("grad", [True, False])
def test_weights_and_teacher_types(td, grad):
    say("weights", td, grad)
    z, u, idx = make(40, 1003, 10, "bf16", 6, td=td)
    w = torch.rand(40, generator=torch.Generator().manual_seed(0))
    w[::5] = 0
    w[7] = -0.5
    z[5] = float("nan")      # weight 0: not looked at
    z[10] = float("inf")
    check(z, u, idx, w=w, grad=grad)


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [777, 33333])
def test_absent_slots_and_empty_rows(V, cd):
    say("absent", V, cd)
    z, u, idx = make(12, V, 20, cd, 7)
    idx[0, 3:] = -1
    idx[1, :] = -1                       # an empty row
    idx[2, ::2] = V                      # outside the vocabulary
    idx[3, :19] = -2 ** 31
    u[4, 5:] = float("-inf")
    u[5, :] = float("-inf")              # an empty row
    z[1] = float("nan")
    idx[6, 1] = V - 1
    idx[6, 2] = 0
    for bits in (32, 64):
        check(z, u, idx, T=0.7, bits=bits)
    far = idx.clone()
    far[7, 4] = 2 ** 40 + 3              # must not be cut to 32 bits
    check(z, u, far, bits=64)


@pytest.mark.parametrize("n,V", [(5, 300), (5, 30000), (70, 30000)])
def test_the_same_index_more_than_once(n, V):
    say("repeated index", n, V)
    z, u, idx = make(n, V, 40, "f32", 8)
    idx[0, :] = 17
    idx[1, 10:30] = idx[1, 5].item()
    idx[2, 39] = idx[2, 0].item()
    check(z, u, idx)


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [500, 40000, 170001])
def test_forbidden_entries(V, cd):
    """-inf and the type's lowest value among the logits."""
    say("forbidden", V, cd)
    z, u, idx = make(4, V, 12, cd, 9)
    top = idx[:, :12]
    z[:, V // 2:] = float("-inf")
    z[1, : V // 3] = torch.finfo(z.dtype).min
    z.scatter_(1, top, torch.randn(4, 12).to(z.dtype))  # the teacher's entries stay allowed
    check(z, u, idx)
    z2 = torch.full((2, V), torch.finfo(z.dtype).min, dtype=z.dtype)  # every entry at the lowest value: uniform
    check(z2, u[:2], idx[:2])
    z2[0, 5] = 1.0
    check(z2, u[:2], torch.full_like(idx[:2], 5))
    big = torch.full((2, V), float(torch.finfo(z.dtype).max), dtype=z.dtype)
    big[:, ::3] = 0
    check(big, u[:2], torch.zeros_like(idx[:2]) + 1)


@pytest.mark.parametrize("V", [500, 40000, 170001])
def test_values_that_are_not_finite(V):
    say("not finite", V)
    z, u, idx = make(6, V, 6, "f32", 10)
    z[0, V - 1] = float("nan")
    z[1, 2] = float("inf")
    z[2, idx[2, 0]] = float("-inf")      # the teacher wants a forbidden entry: loss +inf, finite gradient
    u[3, 1] = float("nan")
    u[4, 0] = float("inf")
    w = torch.ones(6)
    kl = torch.empty(6, device="cuda")
    loss, dz = qn.distill_loss_grad(z.cuda(), u.cuda(), idx.cuda(), weight=w.cuda(), row_kl=kl)
    kl, dz = to_np(kl), to_np(dz)
    assert np.isnan(kl[[0, 1, 3, 4]]).all() and kl[2] == np.inf and np.isfinite(kl[5])
    assert np.isnan(loss.item())
    assert np.isnan(dz[0]).all() and np.isnan(dz[1]).all() and np.isfinite(dz[2]).all() and np.isfinite(dz[5]).all()
    assert np.isnan(dz[3][to_np(idx)[3]]).all() and np.isnan(dz[4][to_np(idx)[4]]).any()


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [257, 32003, 99999, 180001])
def test_in_place_and_padded_rows(V, cd):
    say("in place, padded", V, cd)
    for pad in (0, 1, 5, 24):
        z, u, idx = make(5, V, 10, cd, V + pad, pad=pad)
        check(z, u, idx, in_place=True)
        check(z, u, idx, dz_pad=3 if pad == 1 else 8)


def test_rows_at_every_alignment():
    say("alignment")
    base = torch.randn(40 + 3 * 1001, dtype=torch.float32).bfloat16().cuda()
    u, idx = torch.randn(3, 4).cuda(), torch.randint(0, 1000, (3, 4)).cuda()
    for shift in range(9):
        z = base[shift:shift + 3 * 1001].view(3, 1001)[:, :1000]
        loss, dz = qn.distill_loss_grad(z, u, idx)
        ref, rdz = qn.distill_loss_grad(z.contiguous(), u, idx)
        assert torch.allclose(loss, ref, rtol=1e-5)
        assert torch.allclose(dz.float(), rdz.float(), rtol=2.0 ** -7, atol=1e-8)


def test_no_rows():
    say("no rows")
    loss, dz = qn.distill_loss_grad(torch.empty(0, 50, device="cuda"), torch.empty(0, 3, device="cuda"),
                                    torch.empty(0, 3, dtype=torch.int64, device="cuda"))
    assert loss.item() == 0.0 and dz.shape == (0, 50)


def test_leading_dims():
    say("leading dims")
    z, u, idx = make(12, 100, 4, "f32", 1)
    loss, dz = qn.distill_loss_grad(z.cuda().view(3, 4, 100), u.cuda().view(3, 4, 4), idx.cuda().view(3, 4, 4))
    l2, d2 = check(z, u, idx)
    assert dz.shape == (3, 4, 100) and torch.equal(dz.view(12, 100), d2) and torch.equal(loss, l2)


@pytest.mark.parametrize("n,V", [(64, 5000), (64, 50000), (65, 50000)])
def test_the_same_bits_every_time(n, V):
    say("deterministic", n, V)
    z, u, idx = make(n, V, 16, "bf16", 2)
    idx[:, 3] = idx[:, 0]  # shares of one index are added in slot order
    idx[:, 9] = idx[:, 0]
    a = qn.distill_loss_grad(z.cuda(), u.cuda(), idx.cuda())
    for _ in range(3):
        b = qn.distill_loss_grad(z.cuda(), u.cuda(), idx.cuda())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_against_differences():
    """fp32 logits, the loss differenced with a step whose own errors are counted: truncation
    h^2 / 6 times the third derivative (below w T), rounding of two losses over 2 h."""
    say("differences")
    z, u, idx = make(2, 11, 4, "f32", 3, spread=1.0)
    w = torch.tensor([0.5, 1.5])
    zc, h = z.cuda(), 2.0 ** -6
    _, dz = qn.distill_loss_grad(zc, u.cuda(), idx.cuda(), weight=w.cuda())
    for i in range(2):
        for j in range(11):
            l = []
            for s in (h, -h):
                zz = zc.clone()
                zz[i, j] += s
                l.append((zz[i, j].item(), qn.distill_loss_grad(zz, u.cuda(), idx.cuda(), weight=w.cuda(),
                                                                need_grad=False)[0].item()))
            num = (l[0][1] - l[1][1]) / (l[0][0] - l[1][0])
            assert abs(num - dz[i, j].item()) <= 1.5 * h * h / 6 + 20 * 2.0 ** -24 * 8 / (2 * h)


@pytest.mark.parametrize("n,V", [(20, 3000), (20, 40000), (100, 40000)])
def test_captured_and_replayed(n, V):
    say("graph", n, V)
    k = 8
    z, u, idx = (t.cuda() for t in make(n, V, k, "bf16", 4))
    w = torch.ones(n, device="cuda")
    dz = torch.empty_like(z)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qn.distill_loss_grad(z, u, idx, weight=w, dlogits=dz)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, _ = qn.distill_loss_grad(z, u, idx, weight=w, dlogits=dz)
    for step in range(4):
        z2, u2, idx2 = make(n, V, k, "bf16", 100 + step)
        z.copy_(z2)
        u.copy_(u2)
        idx.copy_(idx2)
        w.copy_(torch.rand(n).round() if step % 2 else torch.rand(n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        l2, d2 = qn.distill_loss_grad(z, u, idx, weight=w)
        assert torch.equal(loss, l2) and torch.equal(dz, d2), "replay %d" % step


def test_python_refusals():
    z = torch.randn(4, 50, device="cuda")
    u, idx = torch.randn(4, 3, device="cuda"), torch.randint(0, 50, (4, 3), device="cuda")
    for call, err in [
        (lambda: qn.distill_loss_grad(z.cpu(), u, idx), ValueError),
        (lambda: qn.distill_loss_grad(z.double(), u, idx), TypeError),
        (lambda: qn.distill_loss_grad(z, u.cpu(), idx), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx.cpu()), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx.short()), TypeError),
        (lambda: qn.distill_loss_grad(z, u.double(), idx), TypeError),
        (lambda: qn.distill_loss_grad(z, u[:, :2], idx), ValueError),
        (lambda: qn.distill_loss_grad(z, u[:3], idx[:3]), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx, weight=torch.ones(3, device="cuda")), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx, weight=torch.ones(4, device="cuda").half()), TypeError),
        (lambda: qn.distill_loss_grad(z, u, idx, temperature=0.0), qn.QloraError),
        (lambda: qn.distill_loss_grad(z, u, idx, dlogits=torch.empty(4, 51, device="cuda")), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx, dlogits=torch.empty(50, 4, device="cuda").t()), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx, dlogits=torch.empty(4, 50, device="cuda").half()), ValueError),
        (lambda: qn.distill_loss_grad(z, u, idx, dlogits=z, need_grad=False), ValueError),
        (lambda: qn.distill_loss_grad(z, torch.randn(4, 1025, device="cuda"),
                                      torch.zeros(4, 1025, dtype=torch.int64, device="cuda")), qn.QloraError),
    ]:
        with pytest.raises(err):
            call()
