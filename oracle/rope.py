"""Per-head RMS norm and rotary positions of q and k, and their gradients (fp64).

Test infrastructure only (see the package docstring).

Source: TensorFold pull request #948, first comment (q/k norm and rotary among
the row kernels around the projections). The page defines neither; these are
the usual definitions. Every pair (a, b) of a head is turned by the angle
positions[row, axis of the pair] * frequency of the pair.
"""

import numpy as np

from .norm import rmsnorm, rmsnorm_backward


def _pair_columns(head_dim, pairs, halves):
    p = np.arange(pairs)
    return (p, pairs + p) if halves else (2 * p, 2 * p + 1)


def _turn(x, positions, inv_freq, pair_axis, halves, sign):
    """x [m, heads, head_dim] turned pair by pair, the rest of a head as it is."""
    first, second = _pair_columns(x.shape[-1], len(pair_axis), halves)
    theta = np.asarray(positions, dtype=np.float64)[:, list(pair_axis)] * np.asarray(inv_freq, dtype=np.float64)
    cos, sin = np.cos(theta)[:, None, :], sign * np.sin(theta)[:, None, :]
    y = x.copy()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., first] * sin + x[..., second] * cos
    return y


def norm_rope(x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps):
    """x [m, heads * head_dim]: the heads normed (gamma None: not) and turned."""
    x = np.asarray(x, dtype=np.float64)
    h = x.reshape(x.shape[0], -1, head_dim)
    n = h if gamma is None else rmsnorm(h, gamma, eps)
    return _turn(n, positions, inv_freq, pair_axis, halves, 1.0).reshape(x.shape)


def norm_rope_backward(dy, x, head_dim, positions, inv_freq, pair_axis, halves, gamma, eps):
    """(dx, dgamma or None)."""
    dy = np.asarray(dy, dtype=np.float64)
    g = _turn(dy.reshape(dy.shape[0], -1, head_dim), positions, inv_freq, pair_axis, halves, -1.0)
    if gamma is None:
        return g.reshape(dy.shape), None
    dx, dgamma = rmsnorm_backward(g, np.asarray(x, dtype=np.float64).reshape(g.shape), gamma, eps, rotate=False)
    return dx.reshape(dy.shape), dgamma
