"""Error bounds of the fp32 arithmetic of the operators around the projections,
from the operations that the kernels do: U is half an fp32 step relative to the
value; a sum of n terms in any order is off by at most (n - 1) U times the sum
of their magnitudes, to first order. The 1.01 covers the higher orders."""

import numpy as np

import oracle

U = 2.0 ** -24        # fp32: torch.finfo(torch.float32).eps / 2
HALF_BF16 = 2.0 ** -8  # bf16: torch.finfo(torch.bfloat16).eps / 2
TINY = 2.0 ** -133     # half the smallest bf16 step: results that small are off by that at most


def group_l1(x):
    """Sum of magnitudes of each element's 256-group."""
    m, k = x.shape
    return np.repeat(np.abs(x).reshape(m, k // 256, 256).sum(axis=2), 256, axis=1)


def inv_rms(t, eps):
    return 1.0 / np.sqrt(np.mean(t * t, axis=-1, keepdims=True) + eps)


def norm_rows(t, gamma, eps, rotate):
    """The normed rows and their bound before the last rounding: t gamma (one
    rounding), 8 butterfly stages on sums of at most the group's magnitudes,
    the row factor (16 squares summed in fp32: 8 steps of the root; its own
    rounding) and the product with it."""
    h = oracle.rmsnorm(t, gamma, eps)
    y = oracle.rotate_groups(h) if rotate else h
    before = 9 * U * group_l1(h) / 16.0 if rotate else U * np.abs(h)
    return y, 1.01 * (before + 11 * U * np.abs(y))


def norm_backward(dy, t, gamma, eps, dsum, rotate, adds):
    """(dx, bound, dgamma, bound) before dx's last rounding. adds: terms that
    one column of dgamma goes through in a row at most."""
    gam = np.ones(t.shape[1]) if gamma is None else gamma
    g = oracle.rotate_groups(dy) if rotate else dy
    eg = 8 * U * group_l1(dy) / 16.0 if rotate else np.zeros_like(dy)
    r = inv_rms(t, eps)
    k = t.shape[1]
    dx, dgamma = oracle.rmsnorm_backward(dy, t, gamma, eps, dsum=dsum, rotate=rotate)
    w = np.abs(gam * g)
    # the mean square: 16 terms a lane, 6 joins, in fp32: 22 U, so 11 U of r;
    # the weighted sum: a product and as many steps
    es1 = (np.abs(gam * t) * eg).sum(axis=1, keepdims=True) + 23 * U * (w * np.abs(t)).sum(axis=1, keepdims=True)
    s1 = np.abs((gam * g * t).sum(axis=1, keepdims=True))
    bound = (r * np.abs(gam) * eg + 15 * U * r * w + np.abs(t) * r ** 3 / k * (es1 + 40 * U * s1)
             + 2 * U * (0 if dsum is None else np.abs(dsum)))
    bdg = (np.abs(t) * r * eg).sum(axis=0) + (15 + adds) * U * (np.abs(g * t) * r).sum(axis=0)
    return dx, 1.01 * bound, dgamma, 1.01 * bdg


def assert_close(got, want, bound, bf16, what):
    """Element by element: the bound of the arithmetic, and the last rounding."""
    half = HALF_BF16 if bf16 else U
    room = bound + half * (np.abs(want) + bound) + TINY
    off = np.abs(got - want)
    bad = ~(off <= room)
    assert not np.any(bad), (f"{what}: {int(bad.sum())} of {bad.size} values out of bounds, worst "
                             f"{float(np.max(off[bad] / room[bad])):.2f} times the bound")


def assert_sum(got, want, magnitudes, terms, what):
    """A sum of exact products in fp32, in any order: element by element at
    most (terms + 4) U times the sum of magnitudes (4: the factors and the
    store)."""
    room = 1.01 * (terms + 4) * U * magnitudes + TINY
    off = np.abs(got - want)
    bad = ~(off <= room)
    assert not np.any(bad), (f"{what}: {int(bad.sum())} of {bad.size} values out of bounds, worst "
                             f"{float(np.max(off[bad] / room[bad])):.2f} times the bound")


def _partner(x, pairs, halves):
    """Magnitude of each element's pair, |a| + |b|; of the element alone past
    the rotated ones. x [m, heads, head_dim]."""
    s = np.abs(x).copy()
    p = np.arange(pairs)
    first, second = (p, pairs + p) if halves else (2 * p, 2 * p + 1)
    s[..., first] = s[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    return s


def rope_forward(x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps):
    """Before the last rounding. Cosines and sines are off by 8 U at most (the
    fraction of a turn in fp32: pi U; sincospif: 4 U); the row factor by 10 U
    (13 steps of a fp32 sum, so 6.5 of the root, and three roundings); a normed
    element by 12 U, and a turned one by three roundings more."""
    y = oracle.norm_rope(x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps)
    h = x.reshape(x.shape[0], -1, head_dim)
    n = h if gamma is None else oracle.rmsnorm(h, gamma, eps)
    return y, 1.01 * (23 * U * _partner(n, len(pair_axis), halves)).reshape(x.shape)


def rope_backward(dy, x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps, adds):
    """(dx, bound, dgamma, bound); g is off by 11 U of its pair, the rest as in
    norm_backward. adds: terms that a column of dgamma goes through in a row."""
    dx, dgamma = oracle.norm_rope_backward(dy, x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps)
    g, _ = oracle.norm_rope_backward(dy, None, head_dim, positions, inv_freq, pair_axis, halves, None, eps)
    shape = (dy.shape[0], -1, head_dim)
    eg = 11 * U * _partner(dy.reshape(shape), len(pair_axis), halves)
    if gamma is None:
        return dx, 1.01 * eg.reshape(dy.shape), None, None
    g, x = g.reshape(shape), x.reshape(shape)
    r = inv_rms(x, eps)
    w = np.abs(gamma * g)
    es = (np.abs(gamma * x) * eg).sum(axis=-1, keepdims=True) + 20 * U * (w * np.abs(x)).sum(axis=-1, keepdims=True)
    s = np.abs((gamma * g * x).sum(axis=-1, keepdims=True))
    bound = r * np.abs(gamma) * eg + 14 * U * r * w + np.abs(x) * r ** 3 / head_dim * (es + 40 * U * s)
    bdg = (np.abs(x) * r * eg).sum(axis=(0, 1)) + (14 + adds) * U * (np.abs(g * x) * r).sum(axis=(0, 1))
    return dx, 1.01 * bound.reshape(dy.shape), dgamma, 1.01 * bdg
