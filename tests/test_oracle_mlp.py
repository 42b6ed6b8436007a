"""The oracles of the 8-bit floating-point product, the gated block and the drawn dropout mask,
pinned by routes of their own."""
import numpy as np
import pytest

import oracle
from oracle import dropout as od, fp8 as of, gated as og


def test_values_are_the_format():
    v = of.values()
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff]) and np.array_equal(v[128:255], -v[:127])
    assert (np.diff(v[:127]) > 0).all()


def test_codes_are_the_nearest_values():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), 2.0 ** rng.uniform(-14, 8, 20000), of.values()[:127],
                        (of.values()[:126] + of.values()[1:127]) / 2, [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    v = v.astype(np.float32).astype(np.float64)
    codes = of.encode(v)
    near = np.abs(of.values()[:127][None, :] - np.abs(v)[:2000, None]).min(axis=1)
    assert np.array_equal(np.abs(of.values()[codes[:2000]] - v[:2000]), near)
    other = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, other)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -127),
                                    (2.0 ** -140, -127), (3.4e38, 120), (448 * 2.0 ** -127, -127)])
def test_exponents(amax, e):
    assert of.exponent(np.float64(np.float32(amax))) == e


def test_blocks_and_products():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 300)) * 10.0 ** rng.integers(-3, 3, (3, 1))
    w = rng.standard_normal((130, 300))
    c, s = of.to_fp8(x, 1)
    assert c.shape == (3, 384) and s.shape == (3, 3) and not c[:, 300:].any()
    back = of.decode(c, s, 1, 300)
    top = np.repeat(np.abs(np.pad(x, ((0, 0), (0, 84)))).reshape(3, 3, 128).max(2), 128, axis=1)[:, :300]
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, top * 2.0 ** -17)).all()
    y, mag = of.product(x, w)
    assert np.linalg.norm(y - x @ w.T) <= 0.05 * np.linalg.norm(x @ w.T) and (np.abs(y) <= mag * (1 + 1e-12)).all()
    x[1, 290] = np.inf
    assert np.isnan(of.product(x, w)[0]).all(axis=1).tolist() == [False, True, False]


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_gate_gradients_are_differences(kind):
    rng = np.random.default_rng(2)
    g, u, dh = (rng.standard_normal(200) * 3 for _ in range(3))
    dg, du = og.backward(g, u, dh, kind)
    h = 1e-5
    assert np.allclose(dg, dh * (og.forward(g + h, u, kind) - og.forward(g - h, u, kind)) / (2 * h), atol=1e-7)
    assert np.allclose(du, dh * (og.forward(g, u + h, kind) - og.forward(g, u - h, kind)) / (2 * h), atol=1e-7)


def test_activations_against_torch():
    torch = pytest.importorskip("torch")
    z = np.linspace(-12, 12, 1001)
    t = torch.from_numpy(z)
    for kind, f in (("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                    ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        assert np.allclose(og.act(z, kind)[0], f(t).numpy(), rtol=1e-12, atol=1e-14)


def test_generator_known_answers():
    """The published answers for the counters and keys of zeros and of ones."""
    assert od.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    f = 0xffffffff
    assert od.philox([f] * 4, [f] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


def test_drawn_mask():
    m, k, seed, off, p = 5, 21, 0x123456789abcdef0, -3, 0.3
    mask = od.drawn_mask(m, k, seed, off, p)
    o = off & ((1 << 64) - 1)
    for i in range(m):
        for j in range(k):
            w = od.philox([j // 8, i, o & 0xffffffff, o >> 32], [seed & 0xffffffff, seed >> 32])
            bits = w[(j % 8) // 2] >> (16 * (j % 2)) & 0xffff
            assert mask[i, j] == (bits >= round(p * 65536))
    assert od.drawn_mask(4, 9, 1, 2, 0.0).all() and od.threshold(0.9999999) == 65535
    big = od.drawn_mask(400, 1000, 7, 8, 0.1)
    assert abs(big.mean() - 0.9) < 5 * (0.09 / big.size) ** 0.5
    assert not np.array_equal(big, od.drawn_mask(400, 1000, 7, 9, 0.1))
