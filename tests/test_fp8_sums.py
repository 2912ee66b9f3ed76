"""The check of the 8-bit matrix instruction's sums (test_fp8_tiles_gpu.py) sees
fewer bits: losses planted on the host."""

import numpy as np
import pytest

import oracle
from tests.fp8_plan import LOST_8BIT


def _aligned_sums(a, b, bits):
    """A block's sums, eight products at a time, each cut at 2^-bits of the largest
    of its eight."""
    p = (a[:, None, :] * b[None, :, :]).reshape(len(a), len(b), 16, 8)
    top = np.abs(p).max(axis=3, keepdims=True)
    step = np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0)))) * 2.0 ** -bits
    return (np.trunc(p / step) * step).sum(axis=(2, 3))


@pytest.mark.parametrize("bits,seen", [(15, False), (13, False), (11, True), (9, True)])
def test_planted_losses(bits, seen):
    rng = np.random.default_rng(5)
    codes = lambda m: oracle.e4m3_value(oracle.quantize_fp8_rows(rng.standard_normal((m, 128)))[0])  # noqa: E731
    a, b, order = codes(40), codes(50), rng.permutation(128)
    lost = np.linalg.norm(_aligned_sums(a, b, bits) - _aligned_sums(a[:, order], b[:, order], bits)) / np.linalg.norm(a @ b.T)
    assert (lost > 2 * LOST_8BIT) == seen, lost
