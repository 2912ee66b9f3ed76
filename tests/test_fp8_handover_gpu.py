"""What the 8-bit float products return goes on to the operators behind them as it
is: results of odd widths."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests.gpu_util import announce, dev, f64, host

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("m,n", [(5, 1163), (300, 1163), (40, 7), (3, 1), (130, 257)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_results_of_odd_widths_go_on(m, n, dtype):
    d = dev()
    announce("product of odd width handed on", m, n, dtype)
    g = torch.Generator(device=d).manual_seed(n)
    a, sa = tp.tp_quantize_fp8(torch.randn((m, 256), device=d, generator=g))
    w, ws = tp.tp_quantize_fp8(torch.randn((n, 256), device=d, generator=g), block_rows=128)
    y = tp.tp_qgemm_fp8(a, sa, w, ws, out_dtype=dtype)
    assert y.shape == (m, n) and y.dtype == dtype
    given = torch.empty((m, n), device=d, dtype=dtype)  # the caller's own, without room behind its rows
    assert tp.tp_qgemm_fp8(a, sa, w, ws, out=given) is given and torch.equal(given, y)

    rng = torch.tensor([3, 4], dtype=torch.int64, device=d)
    keep = oracle.drop_keep(3, 4, m, n, 0.25)
    out = tp.tp_dropout(y, 0.25, rng, residual=y)
    assert np.array_equal(f64(out), oracle.dropout(f64(y), keep, 0.25, f64(y), dtype == BF16))
    q, s, qt, st = tp.tp_quantize_fp8(y, want="both")
    for got, want in (((q, s), oracle.quantize_fp8_rows(f64(y))), ((qt, st), oracle.quantize_fp8_cols(f64(y)))):
        assert np.array_equal(host(got[0].view(torch.uint8)), want[0]) and np.array_equal(host(got[1]), want[1])
