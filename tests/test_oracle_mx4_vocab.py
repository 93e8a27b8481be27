"""Pins of the float64 oracles of the MX4 codec and of the losses over the
vocabulary: hand-worked blocks, brute force, invariants and differences."""

import numpy as np
import pytest

from oracle import mx4, vocab


def test_mx4_ties_go_to_the_even_code_and_large_values_clip():
    x = np.zeros((1, 32))
    # max 7.5 -> s = 0: halfway points of every pair of levels, then the clip
    x[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5]
    code, byte = mx4.quantize(x)
    assert byte.tolist() == [[127]]
    assert code[0, :9].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    code, _ = mx4.quantize(-x)
    assert code[0, :9].tolist() == [8, 10, 10, 12, 12, 14, 14, 15, 15]


def test_mx4_scale_range():
    x = np.zeros((5, 32))
    x[1, 3], x[2, 3], x[3, 3], x[4, 3] = 2.0 ** -149, 2.0 ** -126, 1.0, np.float64(np.finfo(np.float32).max)
    _, byte = mx4.quantize(x)
    assert byte[:, 0].tolist() == [0, 0, 0, 125, 252]
    assert mx4.quantized(x)[1, 3] == 0.0 and mx4.quantized(x)[3, 3] == 1.0
    x[4, 3] = np.inf
    assert np.isnan(mx4.quantized(x)[4]).all() and not np.isnan(mx4.quantized(x)[:4]).any()


def test_mx4_nearest_by_brute_force_and_idempotent():
    g = np.random.default_rng(1)
    x = g.standard_normal((20, 96)) * np.exp2(g.integers(-20, 20, (20, 1)))
    code, byte = mx4.quantize(x)
    v = mx4.values(code, byte)
    grid = np.concatenate((-mx4.LEVELS, mx4.LEVELS))
    for r in range(20):
        for c in range(96):
            allowed = grid * 2.0 ** (int(byte[r, c // 32]) - 127)
            assert abs(v[r, c] - x[r, c]) == np.abs(allowed - x[r, c]).min()
    assert np.array_equal(mx4.quantized(v), v)


def test_mx4_layout():
    g = np.random.default_rng(2)
    code = g.integers(0, 16, (3, 288)).astype(np.uint8)
    byte = g.integers(0, 255, (3, 9)).astype(np.uint8)
    c, s = mx4.lay_out(code, byte)
    assert c.shape == (3, 256) and s.shape == (2, 3, 8)
    for r, k in ((0, 0), (1, 31), (2, 257), (0, 287)):
        assert (c[r, k // 2] >> (4 * (k % 2))) & 15 == code[r, k]
        assert s[k // 256, r, k % 256 // 32] == byte[r, k // 32]
    assert not c[:, 144:].any() and not s[1, :, 1:].any()


def _numeric(f, z, h=1e-5):
    d = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        if not np.isfinite(z[i]):
            continue
        a, b = z.copy(), z.copy()
        a[i] += h
        b[i] -= h
        d[i] = (f(a) - f(b)) / (2 * h)
    return d


def test_logprobs_gradient_against_differences():
    g = np.random.default_rng(3)
    z = g.standard_normal((4, 9)) * 2
    z[1, 4] = -np.inf
    t = np.array([2, 8, -100, 0])
    gl, gh = g.standard_normal(4), g.standard_normal(4)

    def f(z):
        lp, h, _, _ = vocab.logprobs(z, t, 0)
        return (lp * gl + h * gh).sum()

    np.testing.assert_allclose(vocab.logprobs_grad(z, t, gl, gh), _numeric(f, z), atol=1e-8)


@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_distill_gradient_against_differences(temperature):
    g = np.random.default_rng(4)
    z = g.standard_normal((4, 9))
    z[1, 4] = -np.inf
    idx = np.array([[0, 3, 8], [1, 2, -1], [5, 5, 6], [-1, 9, -1]])
    val = g.standard_normal((4, 3))
    w = g.standard_normal(4)
    loss, d = vocab.distill(z, idx, val, temperature, w)
    np.testing.assert_allclose(d, _numeric(lambda z: (vocab.distill(z, idx, val, temperature, w)[0] * w).sum(), z),
                               atol=1e-8)
    assert loss[3] == 0 and not d[3].any()


def test_distill_is_zero_for_a_student_that_equals_the_teacher():
    g = np.random.default_rng(5)
    z = g.standard_normal((3, 6))
    loss, d = vocab.distill(z, np.tile(np.arange(6), (3, 1)), z, 2.0, np.ones(3))
    np.testing.assert_allclose(loss, 0, atol=1e-15)
    np.testing.assert_allclose(d, 0, atol=1e-15)


def test_flat_rows_and_order_of_equal_words():
    z = np.zeros((2, 50))
    z[1] = np.finfo(np.float32).min
    lp, h, tl, ti = vocab.logprobs(z, np.array([7, 7]), 5)
    np.testing.assert_allclose(lp, -np.log(50))
    np.testing.assert_allclose(h, np.log(50))
    assert ti.tolist() == [[0, 1, 2, 3, 4]] * 2
