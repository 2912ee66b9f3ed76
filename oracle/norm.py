"""Residual addition and RMS norm in front of a projection, and its gradients
(fp64).

Test infrastructure only (see the package docstring).

Sources: TensorFold pull request #948, first comment (RMSNorm and the residual
among the row kernels around the projections, bf16 activations between
operations); tensai docs, "画像生成", sections "幅とメモリ" and "GPU" (the
product's input is rotated per 256 columns and quantized on the device).

The page names the norm without defining it; this is its usual definition:
h = t * gamma / sqrt(mean(t^2) + eps). The residual stream is an fp32 sum held
in the stream's type. The gradient takes the quantization as the identity.
"""

import numpy as np

from .hadamard import rotate_groups
from .quantize import bf16_round


def stream_sum(x, residual, bf16):
    """The new residual stream: fp32(x + residual), rounded once more to bf16
    where the stream is bf16. Returned as fp64."""
    t = (np.asarray(x, dtype=np.float32) + np.asarray(residual, dtype=np.float32)).astype(np.float64)
    return bf16_round(t) if bf16 else t


def _inv_rms(t, eps):
    return 1.0 / np.sqrt(np.mean(t * t, axis=-1, keepdims=True) + eps)


def rmsnorm(t, gamma, eps):
    """t * gamma / sqrt(mean(t^2) + eps), gamma None: ones."""
    t = np.asarray(t, dtype=np.float64)
    h = t * _inv_rms(t, eps)
    return h if gamma is None else h * np.asarray(gamma, dtype=np.float64)


def rmsnorm_backward(dy, t, gamma, eps, dsum=None, rotate=True):
    """(dx, dgamma): dy is the gradient of the normed (rotated) rows, dsum the
    gradient that reaches the stream from behind."""
    dy = np.asarray(dy, dtype=np.float64)
    t = np.asarray(t, dtype=np.float64)
    g = rotate_groups(dy) if rotate else dy
    r = _inv_rms(t, eps)
    w = g if gamma is None else g * np.asarray(gamma, dtype=np.float64)
    dx = r * w - t * r ** 3 * np.mean(w * t, axis=-1, keepdims=True)
    if dsum is not None:
        dx = dx + np.asarray(dsum, dtype=np.float64)
    return dx, np.sum(g * t * r, axis=tuple(range(t.ndim - 1)))
