"""The gradients of a product that no token went through: an empty dx and a dw of
zeros, from the codes that the quantizer returns for no rows."""

import pytest
import torch

import int4_quantized_gemm_amd as tp
from tests.gpu_util import announce, dev

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_no_tokens(dtype):
    d = dev()
    announce("gradients of no tokens", dtype)
    n, k = 300, 512
    w, ws, wt, wst = tp.tp_quantize_fp8(torch.ones((n, k), device=d), block_rows=128, want="both")
    x, dy = torch.zeros((0, k), device=d, dtype=dtype), torch.zeros((0, n), device=d, dtype=dtype)
    a, sa, at, sat = tp.tp_quantize_fp8(dy, want="both")
    xt, sxt = tp.tp_quantize_fp8(x, want="cols")
    assert tp.tp_qgemm_fp8(a, sa, wt, wst).shape == (0, k)
    dw = tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out_dtype=dtype)
    assert dw.shape == (n, k) and dw.dtype == dtype and torch.all(dw == 0)

    # into the caller's buffer, on another stream, and nothing around it
    wide = torch.full((n + 2, k + 8), float("nan"), device=d, dtype=dtype)
    out = wide[1:-1, 4:4 + k]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out=out, stream=side) is out
    side.synchronize()
    assert torch.all(out == 0)
    out[:] = float("nan")
    assert torch.all(torch.isnan(wide))

    # captured and replayed over what was written in between
    again = torch.ones((n, k), device=d, dtype=dtype)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out=again)
    for v in (1.0, 2.0, 3.0):
        again.fill_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.all(again == 0)


def test_no_tokens_still_refused():
    """What is wrong without tokens too."""
    d = dev()
    at, xt = torch.zeros((300, 0), device=d).to(F8), torch.zeros((512, 0), device=d).to(F8)
    sat, sxt = torch.zeros((0, 300), device=d), torch.zeros((0, 512), device=d)
    assert tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1).shape == (300, 512)
    for bad in (lambda: tp.tp_qgemm_fp8(at, sat[:, :299], xt, sxt, b_block_rows=1),
                lambda: tp.tp_qgemm_fp8(at, sat, xt, sxt[:, :511], b_block_rows=1),
                lambda: tp.tp_qgemm_fp8(at, sat, xt, sxt),
                lambda: tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out=torch.zeros((300, 511), device=d))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out_dtype=torch.float16)
    with pytest.raises((ValueError, tp.TPError)):
        tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=64)
