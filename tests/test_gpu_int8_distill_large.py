"""Calls whose arrays pass 2^31 elements or 2^32 bytes: the rows behind those offsets against the
oracle, or against a call on just those rows."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from oracle import int8 as oi
from parity import say, to_np
from test_gpu_int8 import check

pytestmark = pytest.mark.gpu


def rows_on_gpu(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)


@pytest.mark.parametrize("m,n,k", [((1 << 31) // 4096 + 300, 64, 4096), ((1 << 31) // 14400 + 300, 14400, 128)])
def test_tokens_and_outputs(m, n, k):
    say("large product", m, n, k)
    x, w = rows_on_gpu(m, k, seed=1), rows_on_gpu(n, k, seed=2, scale=0.02)
    y = qn.linear_int8(qn.quantize_int8(w), x)
    codes, scale = oi.rows_to_int8(to_np(w))
    at = np.r_[0:4, m // 2:m // 2 + 4, m - 310:m - 290, m - 4:m]
    idx = torch.from_numpy(at).cuda()
    ref, mag = oi.product(to_np(x[idx]), codes, scale)
    check(y[idx], ref, mag, "bf16")


@pytest.mark.parametrize("m", [60, 3000, 12000])
def test_weights_of_experts(m):
    E, n, k = 40, 14336, 4096  # 2.3e9 codes
    say("large experts", m)
    w = torch.empty(E, n, k, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = rows_on_gpu(n, k, seed=10 + e, scale=0.02)
    q = qn.quantize_int8(w)
    x = rows_on_gpu(m, k, seed=3)
    off = np.linspace(0, m, E + 1).astype(np.int32)
    y = qn.linear_int8_experts(q, x, torch.from_numpy(off).cuda())
    for e in (0, E - 3, E - 1):
        one = qn.quantize_int8(w[e])
        assert torch.equal(one.codes[0], q.codes[e]) and torch.equal(one.scale[0], q.scale[e])
        part = slice(int(off[e]), int(off[e + 1]))
        assert torch.equal(y[part], qn.linear_int8(one, x[part]))


def test_logits():
    n, V, k = (1 << 31) // 128000 + 300, 128000, 16
    say("large distillation", n, V)
    z = rows_on_gpu(n, V, seed=4, scale=3.0)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.randint(0, V, (n, k), generator=g, device="cuda")
    u = torch.randn(n, k, generator=g, device="cuda")
    w = torch.rand(n, generator=g, device="cuda")
    kl = torch.empty(n, device="cuda")
    loss, dz = qn.distill_loss_grad(z, u, idx, weight=w, row_kl=kl)
    assert abs(loss.item() - (w.double() * kl.double()).sum().item()) <= 2.0 ** -23 * loss.item()
    for at in (slice(0, 20), slice(n - 320, n - 280), slice(n - 20, n)):
        part = torch.empty(at.stop - at.start, device="cuda")
        _, dp = qn.distill_loss_grad(z[at], u[at], idx[at], weight=w[at].contiguous(), row_kl=part)
        # two runs, each within u (8 A + V / 256 + 64) of the probabilities (A < 40), each
        # gradient rounded to bf16 once
        rel = 2 * 2.0 ** -24 * (8 * 40 + V / 256 + 64)
        assert torch.allclose(kl[at].double(), part.double(), rtol=rel, atol=40 * rel)
        assert ((dz[at].float() - dp.float()).abs() <= 2.0 ** -7 * dp.float().abs() + 2 * rel).all()


# A launch takes fewer than 2^32 threads: more rows, tokens or channels than one launch has.
def test_more_channels_than_one_launch_takes():
    n, k = (1 << 29) + 100003, 1
    say("channels", n)
    w = rows_on_gpu(n, k, seed=6)
    q = qn.quantize_int8(w)
    at = torch.tensor([0, 1, (1 << 25) - 1, 1 << 25, 1 << 26, (1 << 26) + 5, n // 2, 1 << 29, n - 100000, n - 2, n - 1],
                      device="cuda")
    codes, scale = oi.rows_to_int8(to_np(w[at]))
    assert np.array_equal(to_np(q.codes[0, at])[:, :k], codes) and not to_np(q.codes[0, at])[:, k:].any()
    assert np.array_equal(to_np(q.scale[0, at]), scale)
    for m in (1, 3):
        x = rows_on_gpu(m, k, seed=7)
        y = qn.linear_int8(q, x)
        ref, mag = oi.product(to_np(x), codes, scale)
        check(y[:, at], ref, mag, "bf16")
        del y


@pytest.mark.parametrize("experts", [None, 3])
def test_more_tokens_than_one_launch_takes(experts):
    m, n, k = (1 << 26) + 333, 2, 8
    say("tokens", m, experts)
    x = rows_on_gpu(m, k, seed=8)
    at = np.r_[0:4, (1 << 25) - 2:(1 << 25) + 2, (1 << 26) - 2:(1 << 26) + 2, m - 4:m]
    idx = torch.from_numpy(at).cuda()
    if experts is None:
        w = rows_on_gpu(n, k, seed=9)
        y = qn.linear_int8(qn.quantize_int8(w), x)
        ref, mag = oi.product(to_np(x[idx]), *oi.rows_to_int8(to_np(w)))
        check(y[idx], ref, mag, "bf16")
        return
    w = rows_on_gpu(experts, n, k, seed=9)
    off = np.array([0, 1 << 25, 1 << 25, m])
    y = qn.linear_int8_experts(qn.quantize_int8(w), x, torch.tensor(off, dtype=torch.int32, device="cuda"))
    for e in (0, 2):
        mine = (at >= off[e]) & (at < off[e + 1])
        ref, mag = oi.product(to_np(x[idx])[mine], *oi.rows_to_int8(to_np(w[e])))
        check(y[idx][torch.from_numpy(mine).cuda()], ref, mag, "bf16")


@pytest.mark.parametrize("n,V,k", [((1 << 26) + 77, 5, 1), ((1 << 24) + 77, 9, 129)])
def test_more_rows_of_logits_than_one_launch_takes(n, V, k):
    say("rows of logits", n, V, k)
    z = rows_on_gpu(n, V, seed=11, scale=2.0)
    u = rows_on_gpu(n, k, seed=12)
    idx = torch.empty(n, k, dtype=torch.int32, device="cuda").random_(0, V)
    w = torch.rand(n, device="cuda") / n
    kl = torch.full((n,), -1.0, device="cuda")
    loss, dz = qn.distill_loss_grad(z, u, idx, weight=w, row_kl=kl)
    total = (w.double() * kl.double()).sum().item()
    assert abs(loss.item() - total) <= 2.0 ** -23 * abs(total)
    assert kl.isfinite().all()
    for a in (0, (1 << 23) - 10, n // 2, (1 << 24) - 10, n - 20):
        s = slice(a, a + 20)
        part = torch.empty(20, device="cuda")
        _, dp = qn.distill_loss_grad(z[s], u[s], idx[s], weight=w[s].contiguous(), row_kl=part)
        rel = 2 * 2.0 ** -24 * (8 * 20 + V / 256 + 64)
        assert torch.allclose(kl[s].double(), part.double(), rtol=rel, atol=20 * rel)
        # each run's entry w T (q - p) is off by rel of w T (q + p) <= 2 w, and rounded to bf16 once
        assert ((dz[s].float() - dp.float()).abs() <= 2.0 ** -7 * dp.float().abs() + 2 * rel * w[s, None]).all()
