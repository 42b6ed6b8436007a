"""The distillation loss where its forms (rows in registers, streamed, in parts) must agree on
values that are not numbers."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn
from parity import TORCH_DT, say, to_np
from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu


# rows, vocabulary, with the gradient: streamed (the loss alone on whole rows, and rows longer than
# the registers), kept in registers, cut into parts
FORMS = [(300, 9001, False), (300, 32000, False), (100, 32003, False), (90, 170007, True), (90, 170007, False), (90, 90001, True),
         (300, 9001, True), (300, 500, True), (300, 500, False), (12, 60003, True), (12, 60003, False)]


@pytest.mark.parametrize("cd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V,grad", FORMS)
def test_nan_among_the_first_entries(n, V, grad, cd):
    """A NaN where a thread has met no number yet: 16 bytes of NaN, one NaN among forbidden
    entries, every thread's first 16 bytes."""
    say("NaN first", n, V, grad, cd)
    z, u, idx = make(n, V, 8, cd, V + n)
    pc = 4 if cd == "f32" else 8
    whole = V // pc * pc
    nan, ninf = float("nan"), float("-inf")
    z[0, :pc] = nan
    z[1, pc:2 * pc] = ninf
    z[1, pc + 1] = nan
    z[2, : min(256 * pc, V // 2)] = nan
    z[3, : V // 2] = ninf
    z[3, 3] = nan
    z[4, :whole] = ninf                    # a number only behind the last whole 16 bytes (or none)
    z[4, 0] = nan
    z[5, whole - pc: whole] = nan
    z[6, : 3 * pc] = ninf                  # no NaN
    idx[:7] = torch.arange(V // 2, V // 2 + 8)
    kl = torch.empty(n, device="cuda")
    loss, dz = qn.distill_loss_grad(z.cuda(), u.cuda(), idx.cuda(), need_grad=grad, row_kl=kl)
    kl = to_np(kl)
    assert np.isnan(kl[:6]).all(), kl[:6]
    assert np.isfinite(kl[6:]).all() and np.isnan(loss.item())
    if grad:
        dz = to_np(dz)
        assert np.isnan(dz[:6]).all() and np.isfinite(dz[6:]).all()
    w = torch.zeros(n)
    w[6:14] = 0.25
    check(z, u, idx, w=w, grad=grad)


@pytest.mark.parametrize("cd", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,grad", [(300, 500, True), (300, 9001, False), (12, 60003, True), (300, 32000, True)])
@pytest.mark.parametrize("T", [0.25, 0.75])
def test_teacher_entries_at_the_lowest_value(T, n, V, grad, cd):
    """A teacher's entry that the student masks with the type's lowest value: kl = T p |lowest|
    and a little, which fp32 holds below T = 1."""
    say("lowest", T, n, V, grad, cd)
    z, u, idx = make(n, V, 8, cd, V + n)
    lowest = torch.finfo(z.dtype).min
    z[0, idx[0, 0]] = lowest
    z[1, idx[1]] = lowest
    z[2, V // 2:] = lowest
    w = torch.zeros(n)
    w[:12] = 1.0 / 64
    check(z, u, idx, T=T, w=w, grad=grad)
