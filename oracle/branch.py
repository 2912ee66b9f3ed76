"""The operators of a pre-norm block's branches in fp64: layer norm and its
gradients, the counter-based dropout, codes in 8-bit floating point with a scale
for each block of 128, and the product of two such matrices.

Test infrastructure only (see the package docstring).

Sources: TensorFold pull request #948, first comment (norm and residual among
the row kernels around the projections); tensai docs, "画像生成", section "GPU"
(the device quantizes each product's activations more finely). The pages give
no formulas for these: layer norm is its usual definition, the generator is
Philox4x32-10 (Salmon and others, "Parallel random numbers: as easy as 1, 2,
3", 2011), e4m3 the 8-bit format of the OCP specification.
"""

import numpy as np

from .hadamard import rotate_groups
from .quantize import bf16_round

BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------- layer norm
def _row(t, eps):
    mean = np.mean(t, axis=-1, keepdims=True)
    d = t - mean
    return d, 1.0 / np.sqrt(np.mean(d * d, axis=-1, keepdims=True) + eps)


def layernorm(t, gamma, beta, eps):
    """(t - mean) / sqrt(variance + eps) * gamma + beta; None: ones, zeros."""
    d, r = _row(np.asarray(t, dtype=np.float64), eps)
    h = d * r
    if gamma is not None:
        h = h * np.asarray(gamma, dtype=np.float64)
    return h if beta is None else h + np.asarray(beta, dtype=np.float64)


def layernorm_backward(dy, t, gamma, eps, dsum=None, rotate=True):
    """(dx, dgamma, dbeta): dy is the gradient of the normed (rotated) rows,
    dsum the gradient that reaches the stream from behind."""
    dy = np.asarray(dy, dtype=np.float64)
    g = rotate_groups(dy) if rotate else dy
    d, r = _row(np.asarray(t, dtype=np.float64), eps)
    n = d * r
    w = g if gamma is None else g * np.asarray(gamma, dtype=np.float64)
    dx = r * (w - np.mean(w, axis=-1, keepdims=True) - n * np.mean(w * n, axis=-1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, dtype=np.float64)
    return dx, np.sum(g * n, axis=0), np.sum(g, axis=0)


# ------------------------------------------------------------------- dropout
def philox4x32_10(counter, key):
    """counter [..., 4], key [2] of 32-bit values -> [..., 4]."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        hp, hq = p >> np.uint64(32), q >> np.uint64(32)
        c = [hq ^ c[1] ^ np.uint64(k[0]), q & low, hp ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1)


def drop_threshold(p):
    return int(np.rint(p * 65536))


def drop_factor(p):
    t = drop_threshold(p)
    return np.float32(65536.0 / (65536 - t)) if t < 65536 else np.float32(0.0)


def drop_keep(seed, offset, m, k, p, rows=None):
    """Whether elements are kept: [m, k], or of the given rows only."""
    rows = np.arange(m) if rows is None else np.asarray(rows)
    runs = (k + 7) // 8
    run = rows.astype(np.uint64)[:, None] * np.uint64(runs) + np.arange(runs, dtype=np.uint64)[None, :]
    ctr = np.empty(run.shape + (4,), dtype=np.uint64)
    ctr[..., 0], ctr[..., 1] = run & np.uint64(0xFFFFFFFF), run >> np.uint64(32)
    offset, seed = int(offset) % 2 ** 64, int(seed) % 2 ** 64
    ctr[..., 2], ctr[..., 3] = offset & 0xFFFFFFFF, offset >> 32
    words = philox4x32_10(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=-1)
    return halves.reshape(len(rows), runs * 8)[:, :k] >= np.uint64(drop_threshold(p))


def dropped(x, keep, p):
    """fp32(x f) where kept, 0 where not (fp32)."""
    x = np.asarray(x, dtype=np.float32)
    if drop_threshold(p) == 0:
        return x
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(keep, x * drop_factor(p), np.float32(0.0)).astype(np.float32)


def dropout(x, keep, p, residual, bf16):
    """drop(x) + residual in fp32, rounded once more to bf16 where the result
    is bf16. Returned as fp64."""
    y = dropped(x, keep, p)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float32)
    y = y.astype(np.float64)
    return bf16_round(y) if bf16 else y


# ------------------------------------------------------- 8-bit floating point
def e4m3_value(codes):
    """What code bytes stand for (0x7f and 0xff: NaN)."""
    codes = np.asarray(codes, dtype=np.uint8)
    e, m = (codes >> 3).astype(np.int64) & 15, (codes & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((codes & 0x7F) == 0x7F, np.nan, v)
    return np.where(codes & 0x80, -v, v)


_VALUES = e4m3_value(np.arange(127))


def e4m3_code(q):
    """The nearest code, the even one of two equally near, at most 448 in
    magnitude; the sign is kept."""
    q = np.asarray(q, dtype=np.float64)
    a = np.minimum(np.abs(q), E4M3_MAX)
    hi = np.clip(np.searchsorted(_VALUES, a), 1, 126)
    lo = hi - 1
    up, down = _VALUES[hi] - a, a - _VALUES[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def _codes(y, axes):
    amax = np.max(np.abs(y), axis=axes, keepdims=True)
    s = (amax / E4M3_MAX).astype(np.float32)
    live = s > 0
    q = y / np.where(live, s, 1).astype(np.float64)
    codes = np.where(live, e4m3_code(q), np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)
    return codes, s


def _padded(x, rows, cols):
    m, k = x.shape
    up = lambda v: -(-v // BLOCK) * BLOCK  # noqa: E731
    out = np.zeros((up(m) if rows else m, up(k) if cols else k))
    out[:m, :k] = x
    return out


def quantize_fp8_rows(x):
    """Codes [m, kp] and scales [kp / 128, m], one for 128 columns of a row."""
    x = _padded(np.asarray(x, dtype=np.float64), False, True)
    c, s = _codes(x.reshape(x.shape[0], -1, BLOCK), 2)
    return c.reshape(x.shape), np.ascontiguousarray(s[:, :, 0].T)


def quantize_fp8_cols(x):
    """Codes of the transpose [k, mp] and scales [mp / 128, k]."""
    return quantize_fp8_rows(np.asarray(x, dtype=np.float64).T)


def quantize_fp8_blocks(x):
    """Codes [m, kp] and scales [mp / 128, kp / 128], one for 128 x 128."""
    m = len(x)
    x = _padded(np.asarray(x, dtype=np.float64), True, True)
    c, s = _codes(x.reshape(x.shape[0] // BLOCK, BLOCK, x.shape[1] // BLOCK, BLOCK), (1, 3))
    return c.reshape(x.shape)[:m], s[:, 0, :, 0]


def qgemm_fp8(a, sa, b, sb, b_block_rows=128):
    """(C, magnitudes) in fp64: sum_g sa[g, i] sb(g, c) sum_q a b and the same
    sum of magnitudes."""
    va = e4m3_value(a) * np.repeat(np.asarray(sa, dtype=np.float64).T, BLOCK, axis=1)
    s = np.asarray(sb, dtype=np.float64)
    if b_block_rows == 1:
        full = np.repeat(s.T, BLOCK, axis=1)
    else:
        full = np.repeat(np.repeat(s, BLOCK, axis=0)[:len(b)], BLOCK, axis=1)
    vb = e4m3_value(b) * full
    return va @ vb.T, np.abs(va) @ np.abs(vb).T
