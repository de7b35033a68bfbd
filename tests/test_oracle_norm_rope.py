"""The oracle of norms with positions against complex arithmetic and against differences."""
import numpy as np
import pytest

from oracle import norm_rope as ON


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, th = rng.standard_normal((5, 24)), rng.standard_normal((5, 4))
    for halves in (False, True):
        got = ON.rotate(x, th, 8, halves)
        z = x[:, 8:16]
        z = z[:, :4] + 1j * z[:, 4:] if halves else z[:, 0::2] + 1j * z[:, 1::2]
        z = z * np.exp(1j * th)
        want = np.concatenate([z.real, z.imag], 1) if halves else np.stack([z.real, z.imag], 2).reshape(5, 8)
        np.testing.assert_allclose(got[:, 8:16], want, atol=1e-14)
        np.testing.assert_array_equal(got[:, :8], x[:, :8])
        np.testing.assert_array_equal(got[:, 16:], x[:, 16:])
        np.testing.assert_allclose(ON.rotate(got, -th, 8, halves), x, atol=1e-14)


def test_angles_of_far_positions():
    # 2^31 - 1 turns and a quarter, and the sum over axes
    pos = np.array([[2 ** 31 - 1], [3]])
    quarter = np.longdouble("6.28318530717958647692528676655900576") * 5 / 4
    th = ON.angles(pos, np.array([[quarter], [0.5]], dtype=np.longdouble))
    want = ((2 ** 31 - 1) * 5 % 4) / 4 * 2 * np.pi + 1.5
    assert abs(np.exp(1j * th[0, 0]) - np.exp(1j * want)) < 1e-8


def test_scores_depend_on_differences_of_positions():
    rng = np.random.default_rng(1)
    q, k, f = rng.standard_normal(16), rng.standard_normal(16), rng.standard_normal((1, 8))
    s = [ON.rotate(q, ON.angles([a], f), 0, False) @ ON.rotate(k, ON.angles([b], f), 0, False) for a, b in ((7, 3), (104, 100))]
    assert abs(s[0] - s[1]) < 1e-12


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_backward_against_differences(halves, weight):
    rng = np.random.default_rng(2)
    x, g, th = rng.standard_normal((3, 24)), rng.standard_normal((3, 24)), rng.standard_normal((3, 4))
    w = rng.standard_normal(24) if weight else None
    f = lambda a, b: float((ON.forward(a, b, 1e-3, th, 8, halves) * g).sum())  # noqa: E731
    dx, dw = ON.backward(x, w, 1e-3, th, 8, halves, g)
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    if weight:
        for i in range(24):
            d = np.zeros(24)
            d[i] = h
            assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[i]) < 1e-7
