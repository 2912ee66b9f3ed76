"""tp_qgemm_fp8 against the fp64 oracle: exactly on codes that are small whole
numbers (every product and sum is exact, so a wrong element, scale or row shows),
and inside the bounds of its sums on quantized random matrices."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests import branch_bounds as R
from tests.gpu_util import announce, dev, f64, host

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
# few rows (1, 2 and 4 fragments, one and several batches of k), the three tiles,
# k split and not, ragged rows and columns, one block of k and many
SHAPES = [(1, 1, 128), (1, 4096, 1280), (2, 17, 256), (16, 130, 4096), (17, 128, 384), (32, 300, 1280), (33, 1163, 1280),
          (64, 129, 640), (64, 2048, 4096), (65, 128, 128), (77, 1163, 1280), (128, 384, 2176), (300, 1000, 512),
          (300, 70, 8192), (513, 640, 256), (1000, 1163, 384)]


def _dev_codes(c, d):
    return torch.from_numpy(np.ascontiguousarray(c)).to(d).view(F8)


def _operands(m, n, k, rows, seed):
    rng = np.random.default_rng(seed)
    a, sa = oracle.quantize_fp8_rows(rng.standard_normal((m, k)))
    w = rng.standard_normal((n, k)) * np.exp(rng.standard_normal((n, 1)))
    b, sb = oracle.quantize_fp8_rows(w) if rows == 1 else oracle.quantize_fp8_blocks(w)
    return a, sa, b, sb


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_random(m, n, k, rows, dtype):
    d = dev()
    announce("tp_qgemm_fp8", m, n, k, rows, dtype)
    a, sa, b, sb = _operands(m, n, k, rows, m + n + k)
    want, mag = oracle.qgemm_fp8(a, sa, b, sb, rows)
    args = (_dev_codes(a, d), torch.from_numpy(sa).to(d), _dev_codes(b, d), torch.from_numpy(sb).to(d))
    got = tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=dtype)
    assert got.dtype == dtype and got.shape == (m, n)
    B.assert_close(f64(got), want, R.product(mag, k, dtype == BF16), dtype == BF16, "C")
    assert torch.equal(got, tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=dtype)), "two runs differ"


def _whole(rng, m, k):
    """Codes of whole numbers -8 .. 8."""
    return oracle.e4m3_code(rng.integers(-8, 9, (m, k)).astype(np.float64))


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("rows", [128, 1])
def test_whole_numbers_are_exact(m, n, k, rows):
    d = dev()
    announce("tp_qgemm_fp8 whole numbers", m, n, k, rows)
    rng = np.random.default_rng(m * n + k)
    a, b = _whole(rng, m, k), _whole(rng, n, k)
    kb = k // 128
    pow2 = lambda *s: (2.0 ** rng.integers(-2, 2, s)).astype(np.float32)  # noqa: E731
    sa = pow2(kb, m)
    sb = pow2(kb, n) if rows == 1 else pow2(-(-n // 128), kb)
    want, mag = oracle.qgemm_fp8(a, sa, b, sb, rows)
    assert mag.max() * 16 < 2 ** 24  # multiples of 1/16 below 2^20: exact in any order
    args = (_dev_codes(a, d), torch.from_numpy(sa).to(d), _dev_codes(b, d), torch.from_numpy(sb).to(d))
    got = tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=F32)
    assert np.array_equal(host(got).astype(np.float64), want), f"{int(np.sum(host(got) != want))} values differ"
    got = tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=BF16)
    assert np.array_equal(f64(got), oracle.bf16_round(want))


@pytest.mark.parametrize("m,n,k,dtype", [(4093, 4091, 256, BF16), (1999, 4093, 128, BF16), (1999, 4093, 128, F32), (4096, 4096, 128, F32)])
def test_large_tiles_exact(m, n, k, dtype):
    """The 256 x 256 and 128 x 128 tiles over full grids with ragged edges, on
    whole numbers; the reference product runs on the device in fp64."""
    d = dev()
    announce("tp_qgemm_fp8 large", m, n, k, dtype)
    g = torch.Generator(device=d).manual_seed(m + n)
    ints = lambda r: torch.randint(-8, 9, (r, k), generator=g, device=d).float()  # noqa: E731
    a, b = ints(m), ints(n)
    sa = 2.0 ** torch.randint(-2, 2, (k // 128, m), generator=g, device=d).float()
    for rows in (128, 1):
        sb = 2.0 ** torch.randint(-2, 2, (k // 128, n) if rows == 1 else (-(-n // 128), k // 128), generator=g, device=d).float()
        full = (sb.t().repeat_interleave(128, 1) if rows == 1 else sb.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1))
        want = (a * sa.t().repeat_interleave(128, 1)).double() @ (b * full).double().t().contiguous()
        got = tp.tp_qgemm_fp8(a.to(F8), sa, b.to(F8), sb, b_block_rows=rows, out_dtype=dtype)
        assert torch.equal(got, want.to(dtype)), f"{int((got != want.to(dtype)).sum())} values differ"


def test_views_and_nothing_around():
    """Codes, scales and results inside larger buffers, results that are not
    16-byte aligned; rows and columns around them stay as they were."""
    d = dev()
    announce("tp_qgemm_fp8 views")
    for m, n, k, dtype in ((5, 130, 384, F32), (5, 130, 384, BF16), (150, 131, 640, F32), (150, 131, 640, BF16), (1000, 1163, 128, BF16)):
        a, sa, b, sb = _operands(m, n, k, 128, 3)
        want, mag = oracle.qgemm_fp8(a, sa, b, sb)

        def inside(x, pad, fill=0x7F):
            buf = np.full((x.shape[0] + 2, x.shape[1] + 2 * pad), fill, dtype=x.dtype)
            buf[1:-1, pad:-pad] = x
            return torch.from_numpy(buf).to(d)

        av, bv = inside(a, 32).view(F8)[1:-1, 32:-32], inside(b, 16).view(F8)[1:-1, 16:-16]
        sav, sbv = inside(sa, 3, np.nan)[1:-1, 3:-3], inside(sb, 1, np.nan)[1:-1, 1:-1]
        c = torch.full((m + 2, n + 7), 4.0, device=d, dtype=dtype)
        out = c[1:-1, 3:3 + n]
        got = tp.tp_qgemm_fp8(av, sav, bv, sbv, out=out)
        assert got is out
        B.assert_close(f64(got), want, R.product(mag, k, dtype == BF16), dtype == BF16, "C")
        out[:] = 4.0
        assert torch.all(c == 4.0)


def test_nan_codes_reach_their_outputs_only():
    d = dev()
    announce("tp_qgemm_fp8 NaN codes")
    for m, n in ((3, 40), (140, 150)):
        a, sa, b, sb = _operands(m, n, 256, 128, 5)
        a[1, 200], b[7, 3] = 0x7F, 0xFF
        for dtype in (F32, BF16):
            got = f64(tp.tp_qgemm_fp8(_dev_codes(a, d), torch.from_numpy(sa).to(d), _dev_codes(b, d), torch.from_numpy(sb).to(d),
                                      out_dtype=dtype))
            bad = np.zeros((m, n), dtype=bool)
            bad[1], bad[:, 7] = True, True
            assert np.array_equal(np.isnan(got), bad)


def test_binding_refuses_wrong_shapes():
    d = dev()
    a = torch.zeros((4, 256), device=d).to(F8)
    s, w, ws = torch.ones((2, 4), device=d), torch.zeros((300, 256), device=d).to(F8), torch.ones((3, 2), device=d)
    assert tp.tp_qgemm_fp8(a, s, w, ws).shape == (4, 300)
    for bad in (lambda: tp.tp_qgemm_fp8(a, s.t(), w, ws), lambda: tp.tp_qgemm_fp8(a, s, w, ws[:2]),
                lambda: tp.tp_qgemm_fp8(a, s, w, ws, b_block_rows=1), lambda: tp.tp_qgemm_fp8(a, s, w[:, :128], ws),
                lambda: tp.tp_dropout(s, 0.1), lambda: tp.tp_layernorm_rotate(torch.zeros((4, 256), device=d), scales=s, out_kind="bf16"),
                lambda: tp.tp_quantize_fp8(s, want="all"), lambda: tp.tp_quantize_fp8(s, want="rows", qt=a)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        tp.tp_qgemm_fp8(a.view(torch.uint8), s, w, ws)
    with pytest.raises(tp.TPError):
        tp.tp_qgemm_fp8(a, s, w, ws, b_block_rows=64)
