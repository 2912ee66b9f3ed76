"""NaN and infinity in what the branch operators turn into codes: they show in the
codes or scales of the rows that hold them, whatever the size of the values beside
them, and leave the other rows as they are."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests.gpu_util import announce, dev, f64, host

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _codes(t):
    return host(t.view(torch.uint8))


def _block_of(x64, rows, cols):
    """Codes and scales of what is left without the NaN; where they were."""
    fine = np.where(np.isnan(x64), 0.0, x64)
    q = {"rows": oracle.quantize_fp8_rows, "cols": oracle.quantize_fp8_cols}
    return q["rows" if rows else "cols"](fine), np.isnan(x64) if rows else np.isnan(x64).T


# values whose scales lie inside and outside the range of the codes' quick way
@pytest.mark.parametrize("size", [1e-44, 1e-36, 1e-29, 1.0, 1e30, 3e38])
def test_nan_has_a_nan_code(size):
    d = dev()
    announce("tp_quantize_fp8 NaN beside values of", size)
    m, k = 150, 300
    rng = np.random.default_rng(1)
    x = (np.clip(rng.standard_normal((m, k)), -1.0, 1.0) * size).astype(np.float32)
    for r, c in ((0, 0), (3, 130), (77, 299), (149, 5), (140, 5)):
        x[r, c] = np.nan
    x[5, 7] = -np.nan
    wide = torch.zeros((m, 304), device=d)[:, :k]
    wide.copy_(torch.from_numpy(x))
    x64 = x.astype(np.float64)
    for want in ("rows", "cols", "both"):
        got = tp.tp_quantize_fp8(wide, want=want)
        for rows, (q, s) in ((True, got[:2]), (False, got[-2:])):
            if want == ("cols" if rows else "rows"):
                continue
            (codes, scales), at = _block_of(x64, rows, not rows)
            assert np.array_equal(host(s), scales)
            q = _codes(q)
            at = np.pad(at, ((0, 0), (0, q.shape[1] - at.shape[1])))
            assert np.all((q[at] & 0x7F) == 0x7F), "a NaN became a number"
            assert np.array_equal(q[~at], codes[~at])
    codes, scales = oracle.quantize_fp8_blocks(np.where(np.isnan(x64), 0.0, x64))
    q, s, qt, _ = tp.tp_quantize_fp8(wide, block_rows=128, want="both")
    at = np.pad(np.isnan(x64), ((0, 0), (0, codes.shape[1] - k)))
    assert np.array_equal(host(s), scales)
    assert np.all((_codes(q)[at] & 0x7F) == 0x7F) and np.array_equal(_codes(q)[~at], codes[~at])
    assert np.array_equal(_codes(qt)[:, :m], _codes(q)[:, :k].T)


@pytest.mark.parametrize("size", [1e-36, 1.0, 1e36])
def test_nan_reaches_the_product(size):
    """Quantized and multiplied: the rows that hold it are NaN, no other is."""
    d = dev()
    announce("NaN through quantizer and product", size)
    m, n, k = 70, 40, 512
    x = torch.from_numpy((np.random.default_rng(2).standard_normal((m, k)) * size).astype(np.float32)).to(d)
    x[3, 100], x[60, 511], x[9, 0] = float("nan"), float("inf"), float("nan")
    w, ws = tp.tp_quantize_fp8(torch.randn((n, k), device=d, generator=torch.Generator(device=d).manual_seed(1)), block_rows=128)
    for rotate in (False, True):
        a, sa = tp.tp_quantize_fp8(x, rotate=rotate)
        if not rotate:
            assert (_codes(a)[60, 511] & 0x7F) == 0x7F and host(sa)[3, 60] == np.inf
        y = f64(tp.tp_qgemm_fp8(a, sa, w, ws))
        bad = np.zeros(m, dtype=bool)
        bad[[3, 9, 60]] = True
        assert not np.any(np.isfinite(y[bad])) and np.all(np.isfinite(y[~bad]))


# rows of one group, rows that share a block, wide rows
@pytest.mark.parametrize("m,k", [(9, 256), (9, 768), (9, 4096), (9, 12288)])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("where", ["x", "residual", "gamma", "beta"])
def test_int8_rows_show_what_is_not_finite(m, k, rotate, where):
    """A row that is not finite has a scale that is not; the others keep their bytes."""
    d = dev()
    announce("tp_layernorm_rotate int8 rows, not finite in", where, m, k, rotate)
    rng = np.random.default_rng(k)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(d)  # noqa: E731
    x, res, gamma, beta = draw(m, k), draw(m, k), draw(k), draw(k)
    call = lambda: tp.tp_layernorm_rotate(x, gamma, beta, residual=res, rotate=rotate, out_kind="i8")  # noqa: E731
    q0, s0, _ = call()
    assert torch.all(torch.isfinite(s0))
    for value, col in ((float("nan"), 0), (float("nan"), k - 1), (float("inf"), 17), (float("nan"), 140)):
        bad = np.zeros(m, dtype=bool)
        if where in ("x", "residual"):
            t = x if where == "x" else res
            bad[[2, 8]] = True
            kept = t[[2, 8], col].clone()
            t[[2, 8], col] = value
        else:
            t = gamma if where == "gamma" else beta
            bad[:] = True
            kept = t[col].clone()
            t[col] = value
        q, s, _ = call()
        assert not np.any(np.isfinite(host(s)[bad])), (value, col)
        assert np.abs(host(q).astype(int)).max() <= 127
        fine = torch.from_numpy(~bad).to(d)
        assert torch.equal(q[fine], q0[fine]) and torch.equal(s[fine], s0[fine])
        if where in ("x", "residual"):
            t[[2, 8], col] = kept
        else:
            t[col] = kept
