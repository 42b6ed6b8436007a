"""The oracles of the 8-bit product and of the distillation loss against their definitions:
values worked out by hand, exact cases and finite differences (CPU)."""
import numpy as np
import pytest

from oracle import distill, int8


def test_codes_by_hand():
    x = np.array([[127.0, -127.0, 63.5, 0.5, 1.5, 2.5, -0.49], [0.0] * 7, [1.0, np.inf, 0, 0, 0, 0, 0],
                  [1.0, np.nan, 0, 0, 0, 0, 0]], np.float32)
    c, s = int8.rows_to_int8(x)
    assert c[0].tolist() == [127, -127, 64, 0, 2, 2, 0] and s[0] == 1.0     # ties to even
    assert c[1].tolist() == [0] * 7 and s[1] == 0.0
    assert np.isnan(s[2]) and np.isnan(s[3]) and not c[2:].any()


def test_codes_of_subnormal_rows_stay_in_range():
    tiny = np.float32(2.0 ** -149)
    for n in (1, 63, 64, 190, 191, 1000):
        c, s = int8.rows_to_int8(np.array([[n * tiny, -tiny, 0.0]], np.float32))
        assert abs(int(c[0, 0])) <= 127 and (s[0] > 0) == (n >= 64)


@pytest.mark.parametrize("k", [1, 127, 128, 1000])
def test_product_error_is_that_of_the_codes(k):
    rng = np.random.default_rng(k)
    x, w = rng.standard_normal((5, k)).astype(np.float32), rng.standard_normal((7, k)).astype(np.float32)
    codes, scale = int8.rows_to_int8(w)
    y, _ = int8.product(x, codes, scale)
    # each factor is off by at most half a step: |x - s c| <= s / 2 (and the rounding of x / s)
    sx = np.abs(x).max(1) / 127 * 0.5001
    sw = np.abs(w).max(1) / 127 * 0.5001
    bound = (np.abs(x).sum(1)[:, None] * sw[None] + np.abs(w).sum(1)[None] * sx[:, None] + k * sx[:, None] * sw[None])
    assert np.all(np.abs(y - x.astype(np.float64) @ w.T.astype(np.float64)) <= bound + 1e-12)


def test_offsets_are_limited_and_never_decrease():
    assert int8.clean_offsets([-3, 5, 2, 99], 10).tolist() == [0, 5, 5, 10]


def test_loss_is_zero_where_the_student_agrees():
    z = np.log(np.array([[0.5, 0.25, 0.25]]))
    loss, kl, dz, _ = distill.loss_grad(z, z, [[0, 1, 2]])
    assert abs(loss) < 1e-15 and np.abs(dz).max() < 1e-15


def test_loss_by_hand():
    # teacher (3/4, 1/4) on entries 2 and 0, student uniform over four
    loss, kl, dz, _ = distill.loss_grad(np.zeros((1, 4)), np.log([[3.0, 1.0]]), [[2, 0]])
    assert np.isclose(loss, 0.75 * np.log(3.0) + 0.25 * np.log(1.0))
    assert np.allclose(dz, [[0.0, 0.25, 0.25 - 0.75, 0.25]])


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_gradient_against_differences(T):
    rng = np.random.default_rng(3)
    n, V, k = 4, 9, 5
    z, u = rng.standard_normal((n, V)), rng.standard_normal((n, k))
    idx = rng.integers(-1, V, (n, k))       # absent slots and repeated indices
    idx[3] = -1                             # a row without a slot
    w = np.array([0.5, 0.0, 2.0, 1.0])
    _, _, dz, _ = distill.loss_grad(z, u, idx, T, w)
    h = 1e-5
    for i in range(n):
        for j in range(V):
            zp, zm = z.copy(), z.copy()
            zp[i, j] += h
            zm[i, j] -= h
            num = (distill.loss_grad(zp, u, idx, T, w)[0] - distill.loss_grad(zm, u, idx, T, w)[0]) / (2 * h)
            assert abs(num - dz[i, j]) < 1e-8
    assert not dz[1].any() and not dz[3].any()


def test_rows_left_out_are_not_looked_at():
    z = np.array([[np.nan, np.inf, 0.0], [0.0, 1.0, 2.0]])
    loss, kl, dz, _ = distill.loss_grad(z, [[0.0], [0.0]], [[0], [1]], weight=[0.0, 1.0])
    assert np.isfinite(loss) and not dz[0].any() and kl[0] == 0
