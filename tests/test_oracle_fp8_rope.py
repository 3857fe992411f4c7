"""The CPU oracles of the 8-bit layers and of the rotary positions, pinned by
independent forms: torch's E4M3 casts, direct sums, complex numbers."""
import numpy as np
import torch

from oracle import fp8, rope


def test_e4m3_grid_matches_the_cast():
    g = np.random.default_rng(0)
    t = np.concatenate([g.uniform(-448, 448, 20000), g.standard_normal(20000) * 2.0 ** g.integers(-12, 8, 20000),
                        np.arange(-448, 449) / 512.0, [0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, -448.0]])
    t = np.clip(t, -448, 448).astype(np.float32)
    assert np.array_equal(fp8.e4m3_round(t), torch.from_numpy(t).to(torch.float8_e4m3fn).double().numpy())


def test_quantise_reconstructs_within_half_a_step():
    """|x - s q| <= 2^-4 |x| + 2^-10 s (half a step of a normal, of a subnormal), plus fp32 roundings."""
    x = np.random.default_rng(1).standard_normal((7, 300)).astype(np.float32).astype(np.float64)
    q, s = fp8.quantize_act(x)
    sv = np.repeat(s.T.astype(np.float64), 128, axis=1)[:, :300]
    assert (np.abs(x - q * sv) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + 2.0 ** -10 * sv * (1 + 1e-6)).all()
    assert np.abs(q).max() == 448
    q, s = fp8.quantize_weight(x.T)
    assert q.shape == (7, 300) and s.shape == (1, 3)
    assert np.abs(q).reshape(7, 300)[:, :128].max() == 448


def test_quantise_edges():
    x = np.zeros((3, 130))
    x[1, 0], x[1, 5], x[2, 129] = np.inf, 3.0, np.nan
    q, s = fp8.quantize_act(x)
    assert (q[0] == 0).all() and s[0, 0] == np.float32(2.0 ** -120)
    assert q[1, 0] == 448 and q[1, 5] == 448 and np.isnan(q[2, 129])


def test_linear_is_the_dequantised_product():
    g = np.random.default_rng(2)
    x, w, b = g.standard_normal((9, 270)), g.standard_normal((270, 150)), g.standard_normal(150)
    qx, sx = fp8.quantize_act(x)
    qw, sw = fp8.quantize_weight(w)
    xd = qx * np.repeat(sx.T.astype(float), 128, axis=1)[:, :270]
    wd = qw * np.repeat(np.repeat(sw.astype(float), 128, 0)[:150], 128, 1)[:, :270]
    y, mag, peak = fp8.linear(qx, sx, qw, sw, b)
    assert np.allclose(y, xd @ wd.T + b, rtol=1e-12, atol=1e-12) and (np.abs(y) <= mag * (1 + 1e-12)).all()
    assert (peak <= mag).all() and (mag - np.abs(b) <= 8 * peak).all()
    # the quantised layer is near the real one: 2^-4 of each operand at most
    assert np.linalg.norm(y - (x @ w + b)) <= 2 * 2.0 ** -4 * np.linalg.norm(np.abs(x) @ np.abs(w))
    y2, _, _ = fp8.grouped_linear(qx, sx, [1, 4, 4, 9], np.stack([qw] * 3), np.stack([sw] * 3), np.stack([b] * 3))
    assert np.isnan(y2[0]).all() and np.allclose(y2[1:], y[1:], rtol=1e-13)


def test_rotation_is_a_complex_product_and_keeps_lengths():
    g = np.random.default_rng(3)
    dims = (4, 6, 2)
    x, pos = g.standard_normal((5, 2, 16)), g.integers(0, 50, (5, 3))
    axis, freq = rope.frequencies(dims, 100.0)
    assert axis.tolist() == [0, 0, 1, 1, 1, 2] and np.allclose(freq[:3], [1, 0.1, 1])
    y = rope.rotate(x, pos, axis, freq)
    z = (x[..., 0:12:2] + 1j * x[..., 1:12:2]) * np.exp(1j * pos[:, axis] * freq)[:, None]
    assert np.allclose(y[..., 0:12:2], z.real) and np.allclose(y[..., 1:12:2], z.imag)
    assert np.array_equal(y[..., 12:], x[..., 12:])
    h = rope.rotate(x, pos, axis, freq, "half")
    assert np.allclose(h[..., :6] ** 2 + h[..., 6:12] ** 2, x[..., :6] ** 2 + x[..., 6:12] ** 2)
    for pairing in ("interleaved", "half"):
        there = rope.rotate(x, pos, axis, freq, pairing)
        assert np.allclose(rope.rotate(there, pos, axis, freq, pairing, inverse=True), x)


def test_relative_positions():
    """The product of a rotated query and key depends on the difference of their positions alone."""
    g = np.random.default_rng(4)
    axis, freq = rope.frequencies((8, 8))
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    dot = lambda a, b: (rope.rotate(q, a, axis, freq) * rope.rotate(k, b, axis, freq)).sum()
    a, b, s = np.array([[3, 9]]), np.array([[7, 2]]), np.array([[11, 5]])
    assert np.isclose(dot(a, b), dot(a + s, b + s))
    assert np.allclose((rope.rms_norm(q, np.ones(16), 0.0) ** 2).mean(), 1.0)
