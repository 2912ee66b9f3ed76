"""Error bounds of the fp32 arithmetic of layer norm, its gradients and the
8-bit float products, from the operations that the kernels do (U and the last
roundings as in block_bounds)."""

import numpy as np

import oracle
from tests.block_bounds import U, group_l1


def _parts(t, eps):
    mean = np.mean(t, axis=1, keepdims=True)
    d = t - mean
    r = 1.0 / np.sqrt(np.mean(d * d, axis=1, keepdims=True) + eps)
    # two subtractions (the first one's result rounds, the second's too), the
    # mean's parts (exact to 2^-48 of it), the row factor's rounding, the product
    err = 4 * U * np.abs(d) * r + 2.0 ** -47 * np.abs(mean) * r
    return d * r, r, err


def layernorm_rows(t, gamma, beta, eps, rotate):
    """The normed rows and their bound before the last rounding: n gamma + beta
    in one rounding, 8 butterfly stages on sums of at most the group's
    magnitudes."""
    n, r, en = _parts(t, eps)
    g = np.ones(t.shape[1]) if gamma is None else gamma
    h = oracle.layernorm(t, gamma, beta, eps)
    eh = np.abs(g) * en + U * (np.abs(h) + np.abs(g) * en)
    if not rotate:
        return h, 1.01 * eh
    return oracle.rotate_groups(h), 1.01 * (group_l1(eh) / 16.0 + 8 * U * group_l1(np.abs(h) + eh) / 16.0)


def layernorm_backward(dy, t, gamma, eps, dsum, rotate, adds):
    """(dx, bound, dgamma, bound, dbeta, bound) before dx's last rounding.
    adds: terms that one column of dgamma and dbeta goes through at most."""
    k = t.shape[1]
    gam = np.ones(k) if gamma is None else gamma
    g = oracle.rotate_groups(dy) if rotate else dy
    eg = 8 * U * group_l1(dy) / 16.0 if rotate else np.zeros_like(dy)
    n, r, en = _parts(t, eps)
    w = gam * g
    ew = np.abs(gam) * eg + U * np.abs(w)
    m1, m2 = np.mean(w, axis=1, keepdims=True), np.mean(w * n, axis=1, keepdims=True)
    # the sums are fp64 sums of the rounded terms; the means round once
    e1 = np.mean(ew, axis=1, keepdims=True) + U * np.abs(m1)
    e2 = np.mean(ew * np.abs(n) + np.abs(w) * en, axis=1, keepdims=True) + 3 * U * np.abs(m2)
    size = np.abs(w) + np.abs(m1) + np.abs(n * m2)
    inner = ew + e1 + np.abs(n) * e2 + np.abs(m2) * en + 2 * U * size
    dx, dgamma, dbeta = oracle.layernorm_backward(dy, t, gamma, eps, dsum=dsum, rotate=rotate)
    bound = r * (inner + 2 * U * size) + 2 * U * (0 if dsum is None else np.abs(dsum))
    bg = (np.abs(n) * eg + np.abs(g) * en).sum(axis=0) + adds * U * np.abs(g * n).sum(axis=0)
    bb = eg.sum(axis=0) + adds * U * np.abs(g).sum(axis=0)
    return dx, 1.01 * bound, dgamma, 1.01 * bg, dbeta, 1.01 * bb


def product(mag, k, bf16):
    """Bound of a product before its last rounding, from its sum of magnitudes.
    fp32 C: exact products, 128 of a block and the blocks' results added in
    fp32, two scale products and a fused add a block. bf16 C: besides, what the
    8-bit matrix instruction drops: of eight products what lies below 2^-15 of
    the largest, 8 2^-15 of the magnitudes at most."""
    return 1.01 * ((128 + k // 128 + 8) * U + (2.0 ** -12 if bf16 else 0.0)) * mag
