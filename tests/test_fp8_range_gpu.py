"""tp_qgemm_fp8 with block scales whose product fp32 does not hold: two tiny ones,
two huge ones over small block sums, blocks of zeros under huge scales. The terms
p sa sb and their sums are ordinary fp32 numbers throughout, and rows and columns
with ordinary scales keep their bytes whatever stands beside them."""

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
PLAIN, TINY, HUGE, ZEROS, SUBNORMAL, NOTHING = range(6)
# log2 of the scales: products reach 2^-140 and 2^130, the sums of their blocks
# 2^22 and (HUGE codes are at most 2^-8) 2^-9
A_EXPONENT = {PLAIN: -6, TINY: -71, HUGE: 96, ZEROS: 126, SUBNORMAL: -135}
B_EXPONENT = {PLAIN: -4, TINY: -69, HUGE: 34, ZEROS: 126, SUBNORMAL: -135}
# few rows with one, two and four fragments; 64 x 128 tiles whole and with k split; 128 x 128; 256 x 256 (bf16)
SHAPES = [(9, 130, 1280), (32, 300, 384), (64, 129, 640), (150, 1163, 640), (300, 70, 8192), (1999, 4093, 384), (4093, 4091, 384)]


def _operand(rng, r, k, exponents, kinds, in_turn=False):
    """Codes [r, k], scales [k / 128, r] and the kind of each row."""
    kind = np.array(kinds)[np.arange(r) % len(kinds) if in_turn else rng.integers(0, len(kinds), r)]
    codes, _ = oracle.quantize_fp8_rows(rng.standard_normal((r, k)))
    small = oracle.e4m3_code(rng.integers(-2, 3, (r, k)) * 2.0 ** -9)
    codes = np.where((kind == HUGE)[:, None], small, codes)
    codes[kind == ZEROS] = 0
    e = np.array([exponents.get(int(v), 0) for v in kind])
    s = np.ldexp(rng.uniform(0.5, 2.0, (k // 128, r)), e[None, :]).astype(np.float32)
    s[:, kind == NOTHING] = 0.0
    return codes.astype(np.uint8), s, kind


def _call(a, sa, b, sb, rows, dtype, d):
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(d)  # noqa: E731
    return tp.tp_qgemm_fp8(t(a).view(F8), t(sa), t(b).view(F8), t(sb), b_block_rows=rows, out_dtype=dtype)


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scale_products_beyond_fp32(m, n, k, rows, dtype):
    d = dev()
    announce("tp_qgemm_fp8 scale products beyond fp32", m, n, k, rows, dtype)
    rng = np.random.default_rng(m + n + k)
    a, sa, ka = _operand(rng, m, k, A_EXPONENT, [PLAIN, PLAIN, TINY, HUGE, ZEROS, SUBNORMAL, NOTHING])
    kinds = [TINY, HUGE, PLAIN, SUBNORMAL, NOTHING]
    if rows == 1:
        b, sb, kb = _operand(rng, n, k, B_EXPONENT, kinds)
    else:  # a kind for each 128 rows of b
        b, s, kb = _operand(rng, -(-n // 128), k, B_EXPONENT, kinds, in_turn=True)
        some, _ = oracle.quantize_fp8_rows(rng.standard_normal((n, k)))
        small = oracle.e4m3_code(rng.integers(-2, 3, (n, k)) * 2.0 ** -9)
        kb = np.repeat(kb, 128)[:n]
        b, sb = np.where((kb == HUGE)[:, None], small, some).astype(np.uint8), np.ascontiguousarray(s.T)
    want, mag = oracle.qgemm_fp8(a, sa, b, sb, rows)
    assert np.all(mag < 2.0 ** 127)
    got = _call(a, sa, b, sb, rows, dtype, d)
    B.assert_close(f64(got), want, R.product(mag, k, dtype == BF16), dtype == BF16, "C")

    # every row of a an ordinary one: the rows that were keep their bytes where b is ordinary too
    ordinary = sa.copy()
    ordinary[:, ka != PLAIN] = 1.0
    again = _call(a, ordinary, b, sb, rows, dtype, d)
    plain = torch.from_numpy(ka == PLAIN).to(d)
    assert torch.equal(again[plain], got[plain]), "rows change with their neighbours' scales"
    strange = sa.copy()
    strange[:, ka == ZEROS] = np.inf
    strange[:, ka == TINY] = np.nan
    again = _call(a, strange, b, sb, rows, dtype, d)
    assert torch.equal(again[plain], got[plain]), "rows change with their neighbours' scales"
    assert np.all(np.isnan(f64(again)[ka == TINY]))


# exponents of scales on either side of where the products change their way, and at the
# ends of fp32
A_EDGES = [-149, -127, -126, -125, -87, -86, -85, -84, -41, -1, 0, 39, 40, 41, 42, 100]
B_EDGES = [-149, -126, -64, -43, -42, -41, -40, -39, 0, 14, 83, 84, 85, 86]


@pytest.mark.parametrize("m,n", [(16, 40), (40, 200), (300, 300), (1999, 4093), (4093, 4091)])
@pytest.mark.parametrize("rows", [128, 1])
def test_scales_at_the_edges(m, n, rows):
    """One block of whole numbers p under powers of two: p 2^e rounded once to fp32
    (subnormal results too), exactly."""
    d = dev()
    announce("tp_qgemm_fp8 scales at the edges", m, n, rows)
    rng = np.random.default_rng(m + n)
    a, b = rng.integers(-8, 9, (m, 128)).astype(np.float64), rng.integers(-8, 9, (n, 128)).astype(np.float64)
    ea = np.array(A_EDGES)[rng.integers(0, len(A_EDGES), m)]
    eb = np.array(B_EDGES)[(np.arange(-(-n // 128)) + m) % len(B_EDGES) if rows == 128 else rng.integers(0, len(B_EDGES), n)]
    e = ea[:, None] + (np.repeat(eb, 128)[:n] if rows == 128 else eb)[None, :]
    p = a @ b.T
    fits = e < 128 - 14  # |p| is at most 2^13
    want = np.ldexp(np.where(fits, p, 0.0), np.where(fits, e, 0)).astype(np.float32)
    power = lambda v: np.ldexp(1.0, v).astype(np.float32)  # noqa: E731
    sa, sb = power(ea)[None, :], power(eb)[:, None] if rows == 128 else power(eb)[None, :]
    for dtype in (F32, BF16):
        got = _call(oracle.e4m3_code(a), sa, oracle.e4m3_code(b), sb, rows, dtype, d)
        ref = torch.from_numpy(want).to(d).to(dtype)
        bad = (got != ref) & torch.from_numpy(fits).to(d)
        assert not torch.any(bad), f"{int(bad.sum())} values differ"
