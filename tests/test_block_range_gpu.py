"""The norms at the far ends of fp32: rows whose elements are finite but whose
sums would leave fp32's range if they were taken in the wrong order. The bounds
are those of ordinary rows: nothing is allowed for the size of the values."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _normal(shape, seed, dtype=F32):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def _large_rows(k, dtype):
    """Rows up to fp32's (bf16's) largest values: a constant one, whose rotated
    groups are 256 times an element before the row factor, one whose groups all
    reach the end of the range, one with a single large element, alternating
    signs, and ordinary rows between them."""
    x = _normal((9, k), k).numpy()
    x[0] = 3e36
    x[2] = np.clip(x[2], -3.3, 3.3) * np.float32(1e38)
    x[3] = 1.0
    x[3, k // 2 + 5] = -3.3e38
    x[5] = 3.3e38
    x[6] = np.where(np.arange(k) % 2 == 0, 2e38, -2e38)
    x[7] *= np.float32(1e35)
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("k", [256, 768, 1024, 4352])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rotate", [True, False])
def test_norm_rows_at_the_end_of_the_range(k, dtype, rotate):
    d = dev()
    announce("tp_rmsnorm_rotate large rows", k, dtype, rotate)
    x = _large_rows(k, dtype)
    # (t gamma itself has to stay in fp32)
    gamma = (0.75 + 0.05 * _normal((k,), k + 1)).clamp(0.5, 1.0)
    for gam in (None, gamma, gamma.to(BF16)):
        g64 = None if gam is None else f64(gam)
        rows = tp.tp_rmsnorm_rotate(x.to(d), None if gam is None else gam.to(d), out_kind="bf16", rotate=rotate)
        want, bound = B.norm_rows(f64(x), g64, 1e-6, rotate)
        B.assert_close(f64(rows), want, bound, True, "rows")
    # as the new stream: the sum, and the rows of it
    res = torch.zeros_like(x)
    rows, t = tp.tp_rmsnorm_rotate(x.to(d), gamma.to(d), residual=res.to(d), out_kind="bf16", rotate=rotate)
    want, bound = B.norm_rows(f64(x), f64(gamma), 1e-6, rotate)
    B.assert_close(f64(rows), want, bound, True, "rows of the stream")
    assert torch.equal(t.cpu(), x)
