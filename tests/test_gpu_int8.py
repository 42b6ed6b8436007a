"""The products in 8-bit integers against the oracle: codes and scales bit by bit, products
within the rounding of their scaling.

Tolerance of a product, element by element: the integer sum is exact; its conversion to fp32,
the two scalings and the bias each round once (2^-24 relative), the result once more into its
type (half a step): |y - ref| <= 2^-24 (3 |scaled sum| + |ref|) + eps / 2 |ref| (+ half the
smallest subnormal), with 10% for the second order."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from oracle import int8 as oi
from parity import TORCH_DT, say, to_np

pytestmark = pytest.mark.gpu


def tensors(m, n, k, cd, seed, experts=None, bias=False):
    g = torch.Generator().manual_seed(seed)
    lead = () if experts is None else (experts,)
    x = (torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))).to(TORCH_DT[cd])
    w = (torch.randn(*lead, n, k, generator=g) * 0.02).to(TORCH_DT[cd])
    b = torch.randn(*lead, n, generator=g).to(TORCH_DT[cd]) if bias else None
    return x, w, b


def check(y, ref, mag, cd, what=""):
    t = TORCH_DT[cd]
    got = to_np(y).astype(np.float64)
    tol = 1.1 * (2.0 ** -24 * (3 * mag + np.abs(ref)) + torch.finfo(t).eps / 2 * np.abs(ref))
    tol += float(torch.finfo(t).tiny) * torch.finfo(t).eps / 2
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, first at %s: %r, expected %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0])


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (5, 128), (2, 129), (7, 1000), (4, 4096), (3, 4104), (2, 14336),
                                       (2, 40001), (1, 131072)])
def test_codes_and_scales(rows, cols, cd):
    say("codes", rows, cols, cd)
    _, w, _ = tensors(1, rows, cols, cd, rows + cols)
    w[0, :] = w[0, :] * 3
    q = qn.quantize_int8(w.cuda())
    codes, scale = oi.rows_to_int8(to_np(w))
    assert q.codes.shape == (1, rows, (cols + 127) // 128 * 128)
    assert np.array_equal(to_np(q.scale)[0], scale)
    assert np.array_equal(to_np(q.codes)[0, :, :cols], codes)
    assert not to_np(q.codes)[0, :, cols:].any()


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
def test_codes_next_to_the_middle(cd):
    """Values at, just below and just above the middle between two codes, under many scales:
    the quotient's rounding to binary32 decides."""
    say("codes: next to the middle", cd)
    g = torch.Generator().manual_seed(5)
    rows = 3000
    amax = torch.randn(rows, generator=g).abs().add(0.01) * torch.pow(10.0, torch.randint(-4, 4, (rows,), generator=g))
    amax = amax.to(TORCH_DT[cd]).float()
    scale = amax / 127
    mid = (torch.arange(-127, 127).float() + 0.5)[None, :] * scale[:, None]
    steps = [mid, torch.nextafter(mid, mid * 2), torch.nextafter(mid, mid * 0)]
    w = torch.cat([amax[:, None]] + steps + [amax[:, None] * 0.5, amax[:, None] * 0.25], 1).to(TORCH_DT[cd])
    w = w.float().clamp(-amax[:, None], amax[:, None]).to(TORCH_DT[cd])
    q = qn.quantize_int8(w.cuda())
    codes, sc = oi.rows_to_int8(to_np(w))
    assert np.array_equal(to_np(q.scale)[0], sc)
    assert np.array_equal(to_np(q.codes)[0, :, :w.shape[1]], codes)
    x = w[:1].cuda()  # the same by the launch that takes one token
    y = qn.linear_int8(qn.quantize_int8(torch.eye(w.shape[1], device="cuda")), x)
    one = to_np(y)[0].astype(np.float64) / float(sc[0])
    assert np.abs(one - codes[0]).max() <= 127 * (torch.finfo(TORCH_DT[cd]).eps + 2.0 ** -22)


def test_codes_at_ties_and_extremes():
    say("codes: ties and extremes")
    t = 2.0 ** -149
    w = torch.zeros(10, 300)
    w[0, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5])      # ties, scale 1
    w[2, 5] = 3.4028234e38
    w[3, :3] = torch.tensor([float("inf"), 1.0, -2.0])
    w[4, 7] = float("nan")
    w[5, :3] = torch.tensor([190 * t, -t, 64 * t])   # the scale rounds to one subnormal step
    w[6, 299] = 62 * t                               # the scale rounds to 0
    w[7, :] = torch.linspace(-1, 1, 300)
    w[8, 0] = -float("inf")
    w[9, :2] = torch.tensor([1e-38, -3e-39])
    q = qn.quantize_int8(w.cuda())
    codes, scale = oi.rows_to_int8(w.numpy())
    assert np.array_equal(to_np(q.scale)[0], scale, equal_nan=True)
    assert np.array_equal(to_np(q.codes)[0, :, :300], codes)


def test_codes_of_strided_rows():
    say("codes: strided rows")
    base = torch.randn(9, 77, dtype=torch.float32).cuda()
    for view in (base[:, 3:60], base[::2, :64], base.t(), base[:, 1:2], base[1:2, 2:9]):
        q = qn.quantize_int8(view)
        codes, scale = oi.rows_to_int8(to_np(view))
        assert np.array_equal(to_np(q.scale)[0], scale)
        assert np.array_equal(to_np(q.codes)[0, :, :view.shape[1]], codes)


SIZES = [(1, 1, 1), (1, 17, 64), (2, 64, 100), (5, 1000, 129), (16, 512, 1024), (17, 130, 4096), (33, 96, 300),
         (64, 257, 2048), (65, 128, 128), (128, 128, 256), (100, 1003, 511), (255, 300, 777), (256, 512, 1024),
         (300, 1030, 2047), (513, 640, 384), (1, 4096, 4096), (16, 14336, 512), (3, 200, 14336), (1030, 1290, 640),
         (1, 40, 16400), (1, 300, 131000), (2, 1001, 640), (15, 9000, 130), (16, 20011, 128), (300, 4099, 129),
         (520, 3001, 257), (600, 4321, 200), (2049, 2051, 130), (61, 500, 9000), (700, 64, 3328),
         (17, 64, 131072), (100, 1001, 2600), (20, 3000, 4000), (3, 2100, 8300), (16, 2049, 8193), (7, 1001, 8400), (500, 1000, 5200), (300, 4096, 7168), (130, 3001, 7200), (250, 700, 14336), (17, 16384, 7300)]


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, cd):
    bias = (m + n) % 2 == 0
    say("product", m, n, k, cd, bias)
    x, w, b = tensors(m, n, k, cd, m + n + k, bias=bias)
    q = qn.quantize_int8(w.cuda())
    y = qn.linear_int8(q, x.cuda(), bias=None if b is None else b.cuda())
    codes, scale = oi.rows_to_int8(to_np(w))
    ref, mag = oi.product(to_np(x), codes, scale, None if b is None else to_np(b))
    check(y, ref, mag, cd)


def test_product_of_a_large_prompt():
    """Whole rounds of the largest tiles and an incomplete one (checked on sampled rows)."""
    m, n, k = 4096 + 57, 4096 + 40, 1024
    say("product", m, n, k)
    x, w, _ = tensors(m, n, k, "bf16", 5)
    y = to_np(qn.linear_int8(qn.quantize_int8(w.cuda()), x.cuda()))
    codes, scale = oi.rows_to_int8(to_np(w))
    rows = np.r_[0:40, 250:260, 2040:2060, m - 70:m]
    ref, mag = oi.product(to_np(x)[rows], codes, scale)
    check(torch.from_numpy(y[rows]).bfloat16(), ref, mag, "bf16")


def test_output_over_the_input_is_refused():
    say("y over x")
    q = qn.quantize_int8(torch.randn(64, 64, device="cuda"))
    x = torch.randn(3, 64, device="cuda")
    kept = x.clone()
    for part in (slice(0, 1), slice(0, 3)):
        with pytest.raises(qn.QloraError):
            qn.linear_int8(q, x[part], out=x[part])
    torch.cuda.synchronize()
    assert torch.equal(x, kept)


def test_a_used_weight_can_be_copied_and_pickled():
    import copy
    import pickle
    say("copies of a weight")
    w, x = torch.randn(70, 130, device="cuda"), torch.randn(2, 130, device="cuda")
    q = qn.quantize_int8(w)
    y = qn.linear_int8(q, x)
    for c in (copy.deepcopy(q), copy.copy(q), pickle.loads(pickle.dumps(q))):
        assert torch.equal(qn.linear_int8(c, x), y)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_largest_sums_do_not_overflow(m):
    """Every code at its limit over the most columns: the sum passes 2^30."""
    k = 131072
    say("largest sums", m)
    x = torch.ones(m, k, dtype=torch.bfloat16)
    x[::2] = -1
    q = qn.quantize_int8(torch.ones(3, k, device="cuda"))
    y = to_np(qn.linear_int8(q, x.cuda()))
    ref, mag = oi.product(to_np(x), np.full((3, k), 127, np.int8), np.full(3, np.float32(1) / np.float32(127)))
    check(torch.from_numpy(y).bfloat16(), ref, mag, "bf16")


@pytest.mark.parametrize("k", [300, 5000])
def test_one_token_that_is_zero_or_not_finite(k):
    say("one special token", k)
    _, w, b = tensors(1, 40, k, "bf16", k, bias=True)
    q = qn.quantize_int8(w.cuda())
    x = torch.zeros(1, k, dtype=torch.bfloat16)
    assert torch.equal(qn.linear_int8(q, x.cuda(), bias=b.cuda()).cpu()[0], b)
    for at, v in ((0, "nan"), (k - 1, "inf"), (k // 2, "-inf")):
        x = torch.ones(1, k, dtype=torch.bfloat16)
        x[0, at] = float(v)
        assert np.isnan(to_np(qn.linear_int8(q, x.cuda(), bias=b.cuda()))).all()
    x = torch.zeros(1, k)
    x[0, 5], x[0, 6] = 190 * 2.0 ** -149, -2.0 ** -149   # a scale of one subnormal step
    qf = qn.quantize_int8(w.float().cuda() * 1e30)
    ref, mag = oi.product(to_np(x), to_np(qf.codes)[0, :, :k], to_np(qf.scale)[0])
    check(qn.linear_int8(qf, x.cuda()), ref, mag, "f32")


@pytest.mark.parametrize("m", [3, 100, 600])
def test_rows_that_are_zero_or_not_finite(m):
    say("special rows", m)
    x, w, b = tensors(m, 200, 300, "bf16", m, bias=True)
    x[0] = 0
    x[1, 17] = float("nan")
    x[m - 1, 299] = float("-inf")
    w[5] = 0
    q = qn.quantize_int8(w.cuda())
    y = qn.linear_int8(q, x.cuda(), bias=b.cuda())
    yn = to_np(y)
    assert np.isnan(yn[1]).all() and np.isnan(yn[m - 1]).all()
    assert np.array_equal(yn[0], to_np(b)) and np.array_equal(yn[2 if m > 3 else 0, 5], to_np(b)[5])
    rows = [i for i in range(m) if i not in (1, m - 1)]
    ref, mag = oi.product(to_np(x)[rows], *oi.rows_to_int8(to_np(w)), to_np(b))
    check(y[rows], ref, mag, "bf16")


def test_a_weight_row_with_nan_gives_a_column_of_nan():
    say("NaN weight row")
    x, w, _ = tensors(20, 60, 90, "f32", 1)
    w[7, 3] = float("nan")
    y = to_np(qn.linear_int8(qn.quantize_int8(w.cuda()), x.cuda()))
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y, 7, axis=1)).all()


@pytest.mark.parametrize("cd", ["f32", "bf16"])
@pytest.mark.parametrize("m", [2, 90, 300])
def test_strided_and_shifted_tokens(m, cd):
    say("strided tokens", m, cd)
    x, w, _ = tensors(m, 130, 515, cd, 9)
    q = qn.quantize_int8(w.cuda())
    ref, mag = oi.product(to_np(x), *oi.rows_to_int8(to_np(w)))
    wide = torch.full((m, 700), float("nan"), dtype=TORCH_DT[cd], device="cuda")
    for shift in (0, 1, 8):
        view = wide[:, shift:shift + 515]
        view.copy_(x)
        check(qn.linear_int8(q, view), ref, mag, cd, "shift %d" % shift)
    check(qn.linear_int8(q, x.cuda().t().contiguous().t()), ref, mag, cd, "transposed")
    y3 = qn.linear_int8(q, x.cuda().reshape(2, m // 2, 515))
    assert y3.shape == (2, m // 2, 130)
    check(y3.reshape(m, 130), ref, mag, cd, "leading dims")


def test_no_tokens():
    say("no tokens")
    q = qn.quantize_int8(torch.randn(8, 16, device="cuda"))
    assert qn.linear_int8(q, torch.empty(0, 16, device="cuda")).shape == (0, 8)
    qe = qn.quantize_int8(torch.randn(2, 8, 16, device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert qn.linear_int8_experts(qe, torch.empty(0, 16, device="cuda"), off).shape == (0, 8)


# ---------------------------------------------------------------------- experts
def check_experts(sizes, n, k, cd, seed, bias=False, before=0, tail=0, offsets=None):
    E = len(sizes)
    m = before + sum(sizes) + tail
    x, w, b = tensors(m, n, k, cd, seed, experts=E, bias=bias)
    q = qn.quantize_int8(w.cuda())
    off = np.r_[0, np.cumsum(sizes)] + before if offsets is None else np.asarray(offsets)
    covered = oi.clean_offsets(off, m)
    x[: covered[0]] = float("nan")  # rows of no expert: whatever they hold
    x[covered[-1]:] = float("inf")
    keep = torch.randn(m, n, generator=torch.Generator().manual_seed(1)).to(TORCH_DT[cd])
    out = keep.cuda()
    y = qn.linear_int8_experts(q, x.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"),
                               bias=None if b is None else b.cuda(), out=out)
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr()
    rows = oi.clean_offsets(off, m)
    left = np.ones(m, bool)
    for e in range(E):
        s = slice(rows[e], rows[e + 1])
        left[s] = False
        if rows[e] < rows[e + 1]:
            ref, mag = oi.product(to_np(x)[s], *oi.rows_to_int8(to_np(w[e])), None if b is None else to_np(b[e]))
            check(y[s], ref, mag, cd, "expert %d" % e)
    assert torch.equal(out.cpu()[torch.from_numpy(left)], keep[torch.from_numpy(left)]), "rows of no expert changed"


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes,n,k,before,tail", [
    ([1], 10, 20, 0, 0),
    ([0, 0, 0], 64, 64, 0, 3),
    ([1, 0, 2, 0, 0, 1], 130, 300, 0, 0),
    ([16, 17, 1, 0, 15], 200, 1024, 2, 5),
    ([64, 65, 63, 1], 128, 512, 0, 1),
    ([0, 300, 0, 5], 257, 130, 0, 130),
    ([128, 129, 127, 0, 256], 300, 384, 7, 0),
    ([700, 0, 3, 400], 520, 200, 0, 33),
    ([30, 0, 64, 7], 130, 5000, 1, 9),
    ([100, 5], 70, 3000, 0, 0),
])
def test_experts(sizes, n, k, before, tail, cd):
    say("experts", sizes, n, k, cd, before, tail)
    check_experts(sizes, n, k, cd, sum(sizes) + n, bias=len(sizes) % 2 == 0, before=before, tail=tail)


@pytest.mark.parametrize("E,m", [(64, 100), (65, 700), (200, 150), (130, 3000)])
def test_many_experts(E, m):
    say("many experts", E, m)
    rng = np.random.default_rng(E)
    sizes = np.bincount(rng.choice(E, m, p=rng.dirichlet(np.full(E, 0.3))), minlength=E)
    check_experts(sizes.tolist(), 70, 200, "bf16", E)


@pytest.mark.parametrize("offsets", [[0, 40, 20, 90, 100], [-5, 10, 500, 30, 2000], [100, 0, 0, 0, 0], [50, 50, 60, 60, 55],
                                     [2 ** 31 - 1, -2 ** 31, 0, 7, 9]])
def test_offsets_out_of_order_or_range(offsets):
    say("offsets", offsets)
    check_experts([25, 25, 25, 25], 90, 150, "bf16", 3, offsets=offsets)


def test_long_runs_of_tiles():
    """Experts with many tiles between experts with one or none (the route is written by lane or
    by the whole wave)."""
    say("long runs of tiles")
    check_experts([1500, 0, 3, 2600, 1, 700, 0, 0, 64, 257], 40, 130, "bf16", 12, before=3, tail=2)
    check_experts([5] * 30 + [900, 0, 1200] + [7] * 60 + [400], 40, 130, "bf16", 13)


def test_all_rows_to_one_expert_of_many():
    say("one expert of many")
    check_experts([0] * 40 + [900] + [0] * 23, 130, 256, "bf16", 4)


def test_experts_agree_with_the_single_product():
    say("experts against the single product")
    x, w, _ = tensors(500, 300, 700, "bf16", 11, experts=3)
    q = qn.quantize_int8(w.cuda())
    y = qn.linear_int8_experts(q, x.cuda(), torch.tensor([0, 4, 200, 500], dtype=torch.int32, device="cuda"))
    for e, (a, b) in enumerate([(0, 4), (4, 200), (200, 500)]):
        one = qn.linear_int8(qn.quantize_int8(w[e].cuda()), x[a:b].cuda())
        assert torch.equal(y[a:b], one)  # exact sums: the same bits whatever kernel forms them


# ------------------------------------------------------------- streams and graphs
def test_runs_on_the_current_stream():
    say("side stream")
    x, w, _ = tensors(300, 520, 1000, "bf16", 2)
    q, xd = qn.quantize_int8(w.cuda()), x.cuda()
    ref = qn.linear_int8(q, xd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        x2 = xd * 1.0
        for _ in range(20):
            x2 = x2 * 1.0
        y = qn.linear_int8(q, x2)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y, ref)


@pytest.mark.parametrize("m", [4, 700])
def test_captured_and_replayed_with_other_rows_and_offsets(m):
    say("graph", m)
    E, n, k = 6, 260, 400
    x, w, _ = tensors(m, n, k, "bf16", 8, experts=E)
    q = qn.quantize_int8(w.cuda())
    q1 = qn.quantize_int8(w[0].cuda())
    xs, off = x.cuda(), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    y1 = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qn.linear_int8_experts(q, xs, off, out=out)
        qn.linear_int8(q1, xs, out=y1)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qn.linear_int8_experts(q, xs, off, out=out)
        qn.linear_int8(q1, xs, out=y1)
    rng = np.random.default_rng(0)
    for step in range(4):
        cuts = np.sort(rng.integers(0, m + 1, E + 1))
        if step == 1:
            cuts[:] = 0
        xs.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(step)).bfloat16())
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = qn.linear_int8_experts(q, xs, off, out=torch.zeros_like(out))
        assert torch.equal(out, want), "replay %d" % step
        assert torch.equal(y1, qn.linear_int8(q1, xs)), "replay %d" % step


# ------------------------------------------------------------------------ refusals
def test_python_refusals():
    q = qn.quantize_int8(torch.randn(8, 16, device="cuda"))
    qe = qn.quantize_int8(torch.randn(2, 8, 16, device="cuda"))
    x = torch.randn(4, 16, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for call, err in [
        (lambda: qn.quantize_int8(torch.randn(8, 16)), ValueError),
        (lambda: qn.quantize_int8(torch.randn(8, device="cuda")), ValueError),
        (lambda: qn.quantize_int8(torch.zeros(8, 16, dtype=torch.int32, device="cuda")), TypeError),
        (lambda: qn.quantize_int8(torch.zeros(1, 131073, device="cuda")), qn.QloraError),
        (lambda: qn.linear_int8(qe, x), ValueError),
        (lambda: qn.linear_int8(qn.Int8Weight(8, 16, q.codes[:, :, :16].contiguous(), q.scale), x), ValueError),
        (lambda: qn.linear_int8(qn.Int8Weight(8, 16, q.codes, q.scale.double()), x), ValueError),
        (lambda: qn.linear_int8(qn.Int8Weight(9, 16, q.codes, q.scale), x), ValueError),
        (lambda: qn.linear_int8(q, x[:, :15]), ValueError),
        (lambda: qn.linear_int8(q, x.cpu()), ValueError),
        (lambda: qn.linear_int8(q, x.double()), TypeError),
        (lambda: qn.linear_int8(q, x, bias=torch.zeros(9, device="cuda")), ValueError),
        (lambda: qn.linear_int8(q, x, bias=torch.zeros(8, device="cuda", dtype=torch.float16)), TypeError),
        (lambda: qn.linear_int8(q, x, out=torch.zeros(4, 9, device="cuda")), ValueError),
        (lambda: qn.linear_int8(q, x, out=torch.zeros(8, 4, device="cuda").t()), ValueError),
        (lambda: qn.linear_int8(q, x, workspace=torch.zeros(8, device="cuda")), ValueError),
        (lambda: qn.linear_int8_experts(qe, x, off.long()), TypeError),
        (lambda: qn.linear_int8_experts(qe, x, off[:2]), ValueError),
        (lambda: qn.linear_int8_experts(qe, x, off.cpu()), ValueError),
        (lambda: qn.linear_int8_experts(qe, x, off, bias=torch.zeros(8, device="cuda")), ValueError),
    ]:
        with pytest.raises(err):
            call()
