"""The references of tests/train_ref.py, held against differences and against
what they have to satisfy, on the CPU."""
import numpy as np
import pytest

import oracle
import train_ref


def test_gated_gradient_against_differences():
    rng = np.random.default_rng(5)
    g, u, dh = rng.standard_normal((3, 400))
    g *= 4
    (dg, _), (du, _) = train_ref.gated_backward(g, u, dh)
    d = 1e-5

    def h(g, u):
        return train_ref.gated(g, u)[0]
    # central differences: off by d^2 / 6 of the third derivative (below 1) and 2^-53 / d
    assert np.allclose(dh * (h(g + d, u) - h(g - d, u)) / (2 * d), dg, rtol=0, atol=1e-9)
    assert np.allclose(dh * (h(g, u + d) - h(g, u - d)) / (2 * d), du, rtol=0, atol=1e-9)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(6)
    T, E, k, H = 5, 3, 2, 4
    ids = rng.integers(-1, E, (T, k))
    R = train_ref.sorted_rows(T, E, k)
    rows, source, _ = train_ref.sort(ids, E, R)
    z, w, dy = rng.standard_normal((R, H)), rng.random((T, k)), rng.standard_normal((T, H))
    dw, _ = train_ref.dweights(dy, z, rows)
    loss = lambda z, w: float((dy * train_ref.combine(z, rows, w)[0]).sum())  # noqa: E731
    for t in range(T):
        for i in range(k):
            step = np.zeros((T, k))
            step[t, i] = 0.5
            assert abs(loss(z, w + step) - loss(z, w - step) - dw[t, i]) < 1e-12      # linear: exact at any step
            if rows[t, i] >= 0:
                step = np.zeros((R, H))
                step[rows[t, i]] = 0.5
                assert source[rows[t, i]] == t * k + i
                assert abs(loss(z + step, w) - loss(z - step, w) - w[t, i] * dy[t].sum()) < 1e-12


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (128, 1, 1), (129, 1, 1), (1000, 60, 4)])
def test_sorted_rows_hold_every_choice(T, E, k):
    R = train_ref.sorted_rows(T, E, k)
    assert R % 512 == 0
    rng = np.random.default_rng(T)
    for _ in range(20):
        ids = rng.integers(0, rng.integers(1, E + 1), (T, k))
        assert train_ref.sort(ids, E, R)[2][-1] <= R


def test_kept_is_exact_under_power_of_two_scales():
    codes = np.tile(np.arange(256, dtype=np.uint8), 3)[: 6 * 128].reshape(6, 128)
    codes[(codes & 0x7F) == 0x7F] = 0
    s = (2.0 ** np.array([-124, -100, 0, 3, 60, 119], dtype=np.float64)).astype(np.float32)[:, None]
    assert np.array_equal(oracle.bf16_to_f64(train_ref.kept(codes, s)), train_ref.dequant(codes, s))
