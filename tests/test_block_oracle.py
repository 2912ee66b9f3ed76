"""Pins of the oracle's operators around the projections: closed forms, plain
loops and gradients against central differences (fp64, CPU)."""

import numpy as np
import pytest

import oracle


def _differences(f, x, step=1e-6):
    """d f / d x for a scalar f, by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + step
        hi = f(x)
        x[i] = keep - step
        lo = f(x)
        x[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


def test_norm_closed_forms():
    t = np.full((1, 256), 3.0)
    assert np.allclose(oracle.rmsnorm(t, None, 1e-300), 1.0, rtol=1e-15)
    t = np.zeros((1, 256))
    t[0, 5] = -2.0  # mean square 4 / 256: h = -16 at 5
    assert np.allclose(oracle.rmsnorm(t, np.arange(256.0), 1e-300)[0, 5], -16.0 * 5.0, rtol=1e-15)
    assert np.all(oracle.rmsnorm(np.zeros((2, 256)), None, 1e-6) == 0.0)
    # eps = 3 mean(t^2) halves the result
    t = np.array([[1.0, -1.0] * 128])
    assert np.allclose(oracle.rmsnorm(t, None, 3.0), t / 2.0, rtol=1e-15)


def test_stream_sum_rounds_to_its_type():
    x = np.float32([1.0, 1.0, 2.0 ** 24])
    res = np.float32([2.0 ** -8, 3 * 2.0 ** -8, 1.0])
    # bf16 steps of 2^-7 above 1: the first is a tie to even (1.0), the second a tie to 1 + 2^-6
    assert oracle.stream_sum(x, res, True).tolist() == [1.0, 1.0 + 2.0 ** -6, 2.0 ** 24]
    assert oracle.stream_sum(x, res, False).tolist() == [1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, 2.0 ** 24]


@pytest.mark.parametrize("rotate", [False, True])
def test_norm_gradient_against_differences(rotate):
    rng = np.random.default_rng(3)
    t = rng.standard_normal((2, 256)) * 2.0
    gamma = 1.0 + 0.2 * rng.standard_normal(256)
    dy, ds = rng.standard_normal((2, 256)), rng.standard_normal((2, 256))

    def loss(t, gamma):
        h = oracle.rmsnorm(t, gamma, 1e-3)
        return np.sum(dy * (oracle.rotate_groups(h) if rotate else h)) + np.sum(ds * t)

    dx, dgamma = oracle.rmsnorm_backward(dy, t, gamma, 1e-3, dsum=ds, rotate=rotate)
    assert np.allclose(dx, _differences(lambda v: loss(v, gamma), t.copy()), rtol=1e-6, atol=1e-6)
    assert np.allclose(dgamma, _differences(lambda v: loss(t, v), gamma.copy()), rtol=1e-6, atol=1e-6)


def test_side_path_gradients_by_loops_and_differences():
    rng = np.random.default_rng(5)
    m, n, k, r, alpha = 3, 5, 256, 2, 1.5
    qa = rng.integers(-127, 128, size=(m, k)).astype(np.int8)
    sa = rng.uniform(0.5, 2.0, size=m).astype(np.float32)
    a, b = rng.standard_normal((r, k)) / 100, rng.standard_normal((n, r))
    dy = rng.standard_normal((m, n))
    t = oracle.lora_down_codes(qa, sa, a)
    for i in range(m):
        for j in range(r):
            assert np.isclose(t[i, j], sum(float(sa[i]) * int(qa[i, q]) * a[j, q] for q in range(k)), rtol=1e-12)
    da, db, dt = oracle.lora_grad_codes(dy, qa, sa, t, b, alpha)

    def loss(a, b):
        return np.sum(dy * alpha * (oracle.lora_down_codes(qa, sa, a) @ b.T))

    assert np.allclose(da, _differences(lambda v: loss(v, b), a.copy(), 1e-4), rtol=1e-7, atol=1e-6)
    assert np.allclose(db, _differences(lambda v: loss(a, v), b.copy(), 1e-4), rtol=1e-7, atol=1e-6)
    assert np.allclose(dt, alpha * dy @ b, rtol=1e-14)
    # trained un-rotated: T = x . (A Q)^T, so the gradient is the codes' domain's times Q
    back, _, _ = oracle.lora_grad_codes(dy, qa, sa, t, b, alpha, rotate=True)

    def loss_rot(a):
        return np.sum(dy * alpha * (oracle.lora_down_codes(qa, sa, oracle.rotate_groups(a)) @ b.T))

    assert np.allclose(back, _differences(loss_rot, a.copy(), 1e-4), rtol=1e-7, atol=1e-6)


def test_rope_closed_forms():
    x = np.zeros((3, 2 * 8))
    x[:, [0, 8]] = 1.0  # the first member of the first pair of both heads
    pos = np.array([[0, 9], [1, 9], [-2, 9]])
    freq = np.array([np.pi / 2, 1.0, 1.0, 1.0])
    # interleaved: the pair is (0, 1); halves: (0, 4); quarter turns of axis 0
    for halves, other in ((False, 1), (True, 4)):
        y = oracle.norm_rope(x, 8, pos, freq, [0, 1, 1, 1], halves, None, 1e-6).reshape(3, 2, 8)
        for row, (c, s) in enumerate([(1, 0), (0, 1), (-1, 0)]):
            for head in range(2):
                assert np.allclose(y[row, head, 0], c, atol=1e-15) and np.allclose(y[row, head, other], s, atol=1e-15)
                assert np.count_nonzero(np.abs(np.delete(y[row, head], [0, other])) > 0) == 0
    # a turn keeps each pair's length, and only positions' differences move q . k
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 8))
    freq = np.array([1.0, 0.3, 0.1, 0.01])

    def dot(i, j):
        at = lambda x, p: oracle.norm_rope(x, 8, [[p]], freq, [0] * 4, True, None, 1e-6)  # noqa: E731
        return float((at(q, i) * at(k, j)).sum())

    assert np.isclose(dot(5, 3), dot(105, 103), rtol=1e-10) and np.isclose(dot(0, 0), float((q * k).sum()))
    # past the rotated pairs a head is passed on, normed
    y = oracle.norm_rope(np.full((1, 16), 2.0), 16, [[7]], [1.0] * 4, [0] * 4, True, np.arange(16.0), 1e-300)
    assert np.allclose(y[0, 8:], np.arange(8.0, 16.0), rtol=1e-15)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_rope_gradient_against_differences(halves, normed):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 2, 32))
    gamma = 1.0 + 0.2 * rng.standard_normal(16) if normed else None
    pos, freq, axis = rng.integers(-50, 50, size=(2, 2)), rng.uniform(0.01, 1.0, 4), [0, 0, 1, 1]

    def loss(x, gamma):
        return np.sum(dy * oracle.norm_rope(x, 16, pos, freq, axis, halves, gamma, 1e-3))

    dx, dgamma = oracle.norm_rope_backward(dy, x, 16, pos, freq, axis, halves, gamma, 1e-3)
    assert np.allclose(dx, _differences(lambda v: loss(v, gamma), x.copy()), rtol=1e-6, atol=1e-7)
    if normed:
        assert np.allclose(dgamma, _differences(lambda v: loss(x, v), gamma.copy()), rtol=1e-6, atol=1e-7)
