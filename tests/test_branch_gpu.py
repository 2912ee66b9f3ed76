"""Dropout, layer norm and its gradients, and the e4m3 quantizers against the
fp64 oracle.

* masks, dropped and summed streams, codes and scales bit for bit: both sides
  take the same decisions (the codes of a normed row differ only where a
  quotient is within about 1e-13 of a tie, which random rows do not reach);
* bf16 rows and gradients inside the bounds of the fp32 arithmetic.
"""

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
SEED, OFFSET = 0x123456789ABCDEF0, 0x0FEDCBA987654321
# one group to 64, rows that share a block (fewer than four groups), rows of one
# to four waves and of sixteen, ragged against both
SHAPES = [(1, 256), (37, 256), (5, 512), (16, 768), (3, 1024), (130, 1280), (7, 3328), (2, 4096), (3, 4352), (2, 12288),
          (1, 16384)]


def _rng(d):
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device=d)


def _draw(m, k, dtype, seed, scale=1.0, shift=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float32) * np.float32(scale) + np.float32(shift)
    x[:, rng.choice(k, size=max(1, k // 200), replace=False)] *= np.float32(30.0)
    return torch.from_numpy(x).to(dtype)


def _vec(k, dtype, seed, about):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((about + 0.1 * rng.standard_normal(k)).astype(np.float32)).to(dtype)


def _padded(t, d, fill=3.0):
    """A device copy inside a wider buffer, its rows 16-byte aligned."""
    per = 16 // t.element_size()
    wide = torch.full((t.shape[0], -(-t.shape[1] // per) * per + 2 * per), fill, dtype=t.dtype, device=d)
    wide[:, per:per + t.shape[1]] = t.to(d)
    return wide[:, per:per + t.shape[1]], wide


def _f8(codes):
    return host(codes.view(torch.uint8))


# ------------------------------------------------------------------- dropout
@pytest.mark.parametrize("m,k", [(1, 1), (1, 8), (3, 7), (5, 9), (64, 1161), (2, 4096), (300, 257)])
@pytest.mark.parametrize("xdt,ydt,res", [(F32, F32, True), (BF16, BF16, True), (BF16, F32, False), (F32, BF16, True), (BF16, BF16, False)])
def test_dropout_bits(m, k, xdt, ydt, res):
    d = dev()
    announce("tp_dropout", m, k, xdt, ydt, res)
    x = _draw(m, k, xdt, seed=m + k)
    r = _draw(m, k, ydt, seed=m + k + 1) if res else None
    xv, _ = _padded(x, d)
    rv = None if r is None else _padded(r, d)[0]
    for p in (0.0, 0.1, 0.5, 1.0, 3e-6):
        got = tp.tp_dropout(xv, p, _rng(d), residual=rv, out_dtype=ydt)
        keep = oracle.drop_keep(SEED, OFFSET, m, k, p)
        want = oracle.dropout(f64(x), keep, p, None if r is None else f64(r), ydt == BF16)
        assert got.dtype == ydt and np.array_equal(f64(got), want), f"p={p}"


def test_dropout_in_place_and_nothing_around():
    d = dev()
    announce("tp_dropout in place")
    m, k = 11, 333
    x = _draw(m, k, F32, seed=1)
    keep = oracle.drop_keep(SEED, OFFSET, m, k, 0.25)
    for alias in ("x", "residual"):
        xv, xb = _padded(x, d)
        rv, rb = _padded(2 * x, d, fill=5.0)
        out = xv if alias == "x" else rv
        got = tp.tp_dropout(xv, 0.25, _rng(d), residual=rv, out=out)
        assert got is out
        assert np.array_equal(f64(got), oracle.dropout(f64(x), keep, 0.25, f64(2 * x), False))
        per = 4
        assert torch.all(xb[:, :per] == 3) and torch.all(xb[:, per + k:] == 3)
        assert torch.all(rb[:, :per] == 5) and torch.all(rb[:, per + k:] == 5)


def test_dropout_special_values_and_gradient():
    """Dropped NaN and infinity are zeros; kept ones stay; the call on a
    gradient is the backward pass; another offset is another mask."""
    d = dev()
    announce("tp_dropout special values")
    x = torch.full((2, 64), float("nan"))
    x[1] = float("inf")
    keep = oracle.drop_keep(SEED, OFFSET, 2, 64, 0.5)
    y = host(tp.tp_dropout(x.to(d), 0.5, _rng(d)))
    assert np.all(y[~keep] == 0) and np.all(np.isnan(y[0][keep[0]])) and np.all(np.isinf(y[1][keep[1]]))
    ones = torch.ones((2, 64), device=d)
    g = host(tp.tp_dropout(ones, 0.5, _rng(d)))
    assert np.array_equal(g, np.where(keep, oracle.drop_factor(0.5), 0))
    other = torch.tensor([SEED, OFFSET + 1], dtype=torch.int64, device=d)
    assert not np.array_equal(host(tp.tp_dropout(ones, 0.5, other)), g)


# ---------------------------------------------------------------- layer norm
def _check(t64, gamma, beta, eps, rotate, kind, got):
    g = None if gamma is None else f64(gamma)
    b = None if beta is None else f64(beta)
    h = oracle.layernorm(t64, g, b, eps)
    if kind == "i8":
        q, s = oracle.quantize_activations_int8(h, rotate=rotate)
        assert np.array_equal(host(got[1]), s), f"{int(np.sum(host(got[1]) != s))} scales differ"
        assert np.array_equal(host(got[0]), q), f"{int(np.sum(host(got[0]) != q))} codes differ"
    elif kind == "fp8":
        hr = oracle.rotate_groups(h) if rotate else h
        q, s = oracle.quantize_fp8_rows(hr)
        assert got[0].dtype == F8
        gs, gq = host(got[1]), _f8(got[0])
        # Values that are exactly zero (images of a group's equal values, sums of
        # rows on a coarse grid) come out as fp64 noise of either sign on either
        # side: 8 stages on sums of at most 256 max|h|, over 16, are off by 2^-46
        # max|h|, and the mean by some 2^-52 of max|t|. There +0 and -0 are one
        # code, and a block of nothing else has any scale of that size.
        noise = 2.0 ** -44 * (np.abs(h).max(axis=1) + np.abs(t64).max(axis=1) / np.sqrt(t64.var(axis=1) + eps))
        lost = 448.0 * s.astype(np.float64) <= noise
        assert np.all((448.0 * gs.astype(np.float64) <= noise)[lost])
        assert np.array_equal(gs[~lost], s[~lost]), f"{int(np.sum(gs != s))} scales differ"
        zero = (np.abs(hr) <= noise[:, None]) & ((gq & 0x7F) == 0) & ((q & 0x7F) == 0)
        bad = (gq != q) & ~zero & ~lost.T.repeat(128, axis=1)
        assert not np.any(bad), f"{int(bad.sum())} codes differ"
    else:
        y, bound = R.layernorm_rows(t64, g, b, eps, rotate)
        B.assert_close(f64(got[0]), y, bound, True, "rows")


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("xdt,sdt,p", [(BF16, BF16, 0.1), (F32, BF16, 0.0), (BF16, F32, 0.5), (F32, None, 0.0), (BF16, None, 0.0),
                                       (F32, F32, 0.1)])
def test_layernorm_shapes_and_types(m, k, xdt, sdt, p):
    d = dev()
    announce("tp_layernorm_rotate", m, k, xdt, sdt, p)
    x = _draw(m, k, xdt, seed=m + k, shift=0.5)
    gdt = BF16 if m % 2 else F32
    gamma, beta = _vec(k, gdt, k, 1.0), _vec(k, gdt, k + 1, 0.0)
    res = None if sdt is None else _draw(m, k, sdt, seed=m + k + 1, scale=2.0)
    t64 = f64(x)
    if res is not None:
        keep = oracle.drop_keep(SEED, OFFSET, m, k, p)
        t64 = oracle.stream_sum(oracle.dropped(f64(x), keep, p), f64(res), sdt == BF16)
    for kind in ("i8", "bf16", "fp8"):
        for rotate in (True, False):
            got = tp.tp_layernorm_rotate(x.to(d), gamma.to(d), beta.to(d), eps=1e-5,
                                         residual=None if res is None else res.to(d), drop_p=p, rng=_rng(d), rotate=rotate,
                                         out_kind=kind)
            got = got if isinstance(got, tuple) else (got,)
            if res is not None:
                assert got[-1].dtype == sdt and np.array_equal(f64(got[-1]), t64), "the new stream differs"
            _check(t64, gamma, beta, 1e-5, rotate, kind, got)


@pytest.mark.parametrize("kind", ["i8", "bf16", "fp8"])
@pytest.mark.parametrize("weights", ["none", "gamma", "beta", "beta f32"])
def test_layernorm_special_rows(kind, weights):
    """Rows of zeros, constant rows, rows far off zero, a single element, rows
    far below eps, huge and subnormal rows; gamma or beta missing."""
    d = dev()
    announce("tp_layernorm_rotate special rows", kind, weights)
    rng = np.random.default_rng(8)
    k = 768
    x = rng.standard_normal((9, k)).astype(np.float32)
    x[1] = 0.0
    x[2] = np.float32(0.1)
    x[3] = 0.0
    x[3, 300] = -3.0
    x[4] *= np.float32(1e-20)
    x[5] = x[5] * np.float32(1e-3) + np.float32(4096.0)
    x[6] *= np.float32(1e18)
    x[7] *= np.float32(1e-39)
    x[8] = np.float32(-7e5)
    xt = torch.from_numpy(x)
    gamma = _vec(k, BF16, 1, 1.0) if weights == "gamma" else None
    beta = _vec(k, F32 if "f32" in weights else BF16, 2, 0.0) if "beta" in weights else None
    for eps in (1e-5, 1e-30):
        for rotate in (True, False):
            got = tp.tp_layernorm_rotate(xt.to(d), None if gamma is None else gamma.to(d), None if beta is None else beta.to(d),
                                         eps=eps, rotate=rotate, out_kind=kind)
            got = got if isinstance(got, tuple) else (got,)
            _check(f64(xt), gamma, beta, eps, rotate, kind, got)
            if beta is None:  # constant rows deviate by nothing
                assert np.all(host(got[0].float())[[1, 2, 8]] == 0)


def test_layernorm_in_place_stream_and_padded_views():
    d = dev()
    announce("tp_layernorm_rotate in place, padded views")
    m, k = 21, 1024
    x, res = _draw(m, k, F32, seed=1), _draw(m, k, F32, seed=2)
    gamma = _vec(k, F32, 3, 1.0)
    t64 = oracle.stream_sum(f64(x), f64(res), False)
    stream = torch.full((m + 2, k + 8), 9.0, device=d)
    stream[1:-1, :k] = res.to(d)
    view = stream[1:-1, :k]
    qb = torch.full((m + 2, k + 64), 7, dtype=torch.uint8, device=d).view(F8)
    sb = torch.full((10, m + 5), -1.0, device=d)
    q, s, t = tp.tp_layernorm_rotate(_padded(x, d)[0], gamma.to(d), residual=view, out_kind="fp8", out=qb[1:-1, 32:32 + k],
                                     scales=sb[1:9, 3:3 + m], sum_out=view)
    assert t is view and np.array_equal(f64(view), t64)
    _check(t64, gamma, None, 1e-5, True, "fp8", (q, s))
    stream[1:-1, :k] = 9.0
    assert torch.all(stream == 9.0)
    around = qb.view(torch.uint8)
    around[1:-1, 32:32 + k] = 7
    assert torch.all(around == 7)
    sb[1:9, 3:3 + m] = -1.0
    assert torch.all(sb == -1.0)


# ----------------------------------------------------------------- gradients
@pytest.mark.parametrize("m,k", SHAPES + [(520, 512), (513, 4096), (40, 5120)])
@pytest.mark.parametrize("ydt,tdt,xdt,ds,p", [(F32, BF16, BF16, True, 0.1), (BF16, BF16, BF16, True, 0.0), (F32, F32, F32, False, 0.0),
                                              (BF16, F32, F32, True, 0.5), (F32, F32, BF16, False, 0.1)])
def test_layernorm_gradients(m, k, ydt, tdt, xdt, ds, p):
    d = dev()
    announce("tp_layernorm_rotate_backward", m, k, ydt, tdt, xdt, ds, p)
    dy = _draw(m, k, ydt, seed=m + k, scale=0.02)
    t = _draw(m, k, tdt, seed=m + k + 1, scale=2.0, shift=1.0)
    dsum = _draw(m, k, xdt, seed=m + k + 2, scale=0.02) if ds else None
    gamma = None if m == 3 else _vec(k, BF16 if m % 2 else F32, k, 1.0)
    g64 = None if gamma is None else f64(gamma)
    for rotate in (True, False):
        dx, branch, dg, db = tp.tp_layernorm_rotate_backward(
            dy.to(d), t.to(d), None if gamma is None else gamma.to(d), eps=1e-5, dsum=None if dsum is None else dsum.to(d),
            drop_p=p, rng=_rng(d), rotate=rotate, dx_dtype=xdt)
        want, bound, wg, bg, wb, bb = R.layernorm_backward(f64(dy), f64(t), g64, 1e-5, None if dsum is None else f64(dsum), rotate,
                                                           m + 40)
        assert dx.dtype == xdt
        B.assert_close(f64(dx), want, bound, xdt == BF16, "dx")
        B.assert_close(f64(dg), wg, bg, False, "dgamma")
        B.assert_close(f64(db), wb, bb, False, "dbeta")
        if p == 0:
            assert branch is None
        else:
            keep = oracle.drop_keep(SEED, OFFSET, m, k, p)
            f = float(oracle.drop_factor(p))
            got = f64(branch)
            assert np.all(got[~keep] == 0)
            B.assert_close(got, np.where(keep, want * f, 0), np.where(keep, (bound + B.U * np.abs(want)) * f, 0), xdt == BF16, "dbranch")
        again = tp.tp_layernorm_rotate_backward(
            dy.to(d), t.to(d), None if gamma is None else gamma.to(d), eps=1e-5, dsum=None if dsum is None else dsum.to(d),
            drop_p=p, rng=_rng(d), rotate=rotate, dx_dtype=xdt, want_dgamma=False)
        assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[3], db)


@pytest.mark.parametrize("k", [512, 4352])
def test_layernorm_gradient_special_rows(k):
    """Constant rows (n is 0), rows far off zero, zero gradients; m == 0 gives
    zero sums; dx in place of dsum and of dy."""
    d = dev()
    announce("tp_layernorm_rotate_backward special rows", k)
    t, dy = f64(_draw(5, k, F32, seed=3)), f64(_draw(5, k, F32, seed=4, scale=0.1))
    t[1], t[2], dy[3] = 0.3, t[2] * 1e-3 + 4096.0, 0.0
    t, dy = (torch.from_numpy(v.astype(np.float32)) for v in (t, dy))
    gamma, ds = _vec(k, BF16, 5, 1.0), _draw(5, k, F32, seed=6, scale=0.1)
    want, bound, wg, bg, wb, bb = R.layernorm_backward(f64(dy), f64(t), f64(gamma), 1e-5, f64(ds), False, 45)
    for alias in (None, "dsum", "dy"):
        dyd, dsd = dy.to(d), ds.to(d)
        out = {None: None, "dsum": dsd, "dy": dyd}[alias]
        if alias == "dy":  # the weights' sums read it: refused with them
            with pytest.raises(tp.TPError):
                tp.tp_layernorm_rotate_backward(dyd, t.to(d), gamma.to(d), eps=1e-5, dsum=dsd, rotate=False, dx=out)
        sums = alias != "dy"
        dx, _, dg, db = tp.tp_layernorm_rotate_backward(dyd, t.to(d), gamma.to(d), eps=1e-5, dsum=dsd, rotate=False, dx=out,
                                                        want_dgamma=sums, want_dbeta=sums)
        B.assert_close(f64(dx), want, bound, False, "dx")
        if not sums:
            continue
        B.assert_close(f64(dg), wg, bg, False, "dgamma")
        B.assert_close(f64(db), wb, bb, False, "dbeta")
    e = torch.zeros((0, k), device=d)
    _, _, dg, db = tp.tp_layernorm_rotate_backward(e, e, gamma.to(d))
    assert torch.all(dg == 0) and torch.all(db == 0)


# ----------------------------------------------------------------- quantizers
QSHAPES = [(1, 1), (1, 128), (3, 7), (16, 256), (17, 130), (128, 128), (129, 257), (300, 384), (5, 2048), (260, 1161)]


def _check_quant(x, m, k, rotate, d, view):
    x64 = f64(x)
    x64 = oracle.rotate_groups(x64) if rotate else x64
    for want in ("rows", "cols", "both"):
        got = tp.tp_quantize_fp8(view, rotate=rotate, want=want)
        if want != "cols":
            q, s = oracle.quantize_fp8_rows(x64)
            assert np.array_equal(host(got[1]), s) and np.array_equal(_f8(got[0]), q), want
        if want != "rows":
            q, s = oracle.quantize_fp8_cols(x64)
            assert np.array_equal(host(got[-1]), s) and np.array_equal(_f8(got[-2]), q), want
        got = tp.tp_quantize_fp8(view, block_rows=128, rotate=rotate, want=want)
        q, s = oracle.quantize_fp8_blocks(x64)
        if want != "cols":
            assert np.array_equal(host(got[1]), s) and np.array_equal(_f8(got[0]), q), "blocks"
        if want != "rows":
            full = np.zeros((k, -(-m // 128) * 128), dtype=np.uint8)
            full[:, :m] = q[:, :k].T
            assert np.array_equal(host(got[-1]), s.T) and np.array_equal(_f8(got[-2]), full), "blocks, transposed"


@pytest.mark.parametrize("m,k", QSHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantizers(m, k, dtype):
    d = dev()
    announce("tp_quantize_fp8", m, k, dtype)
    x = _draw(m, k, dtype, seed=m + k)
    x[0] = 0
    view, _ = _padded(x, d)
    for rotate in ((False, True) if k % 256 == 0 else (False,)):
        _check_quant(x, m, k, rotate, d, view)


def test_quantizer_ties_and_extreme_blocks():
    """Scales of one: every midpoint of the format goes to the even code, its
    neighbours in fp32 to the nearer one; blocks with subnormal and zero scales,
    huge blocks."""
    d = dev()
    announce("tp_quantize_fp8 ties")
    v = oracle.e4m3_value(np.arange(127))
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    rows = [np.concatenate([[448.0, -448.0], mid]), np.concatenate([[448.0, 0.0], np.nextafter(mid, np.float32(1e9))]),
            np.concatenate([[-448.0, 0.0], -np.nextafter(mid, np.float32(0))])]
    rng = np.random.default_rng(3)
    for scale in (1e-36, 2e-38, 1e-40, 3e-43, 1.4e-45, 1e30, 7e37):
        with np.errstate(under="ignore"):
            rows.append((rng.standard_normal(128) * scale).astype(np.float32))
    # scales that are no powers of two, and values at exact ties of them
    s = np.float32(448 * 3) / np.float32(448)
    rows.append(np.concatenate([[448 * s, 0], mid * s]).astype(np.float32))
    x = np.stack([r[:128] for r in rows]).astype(np.float32)
    xt = torch.from_numpy(x)
    _check_quant(xt, x.shape[0], 128, False, d, xt.to(d))
    q, sc = tp.tp_quantize_fp8(xt.to(d))
    assert host(sc)[0, 0] == 1.0
    got = _f8(q)[0, 2:] & 0x7F
    assert np.all(got % 2 == 0), "a midpoint went to an odd code"


def test_quantizer_nothing_around_and_row_zero():
    d = dev()
    announce("tp_quantize_fp8 padded outputs")
    m, k = 77, 200
    x = _draw(m, k, BF16, seed=9)
    bufs = [torch.full(s, 9, dtype=torch.uint8, device=d) for s in ((m + 2, 288), (k + 2, 160))]
    sb = [torch.full(s, -1.0, device=d) for s in ((4, m + 3), (3, k + 3))]
    q, s, qt, st = tp.tp_quantize_fp8(_padded(x, d)[0], want="both", q=bufs[0].view(F8)[1:-1, 16:272], scales=sb[0][1:3, 1:1 + m],
                                      qt=bufs[1].view(F8)[1:-1, 16:144], scales_t=sb[1][1:2, 2:2 + k])
    for got, want in (((q, s), oracle.quantize_fp8_rows(f64(x))), ((qt, st), oracle.quantize_fp8_cols(f64(x)))):
        assert np.array_equal(_f8(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    bufs[0][1:-1, 16:272], bufs[1][1:-1, 16:144] = 9, 9
    sb[0][1:3, 1:1 + m], sb[1][1:2, 2:2 + k] = -1.0, -1.0
    assert all(torch.all(b == 9) for b in bufs) and all(torch.all(b == -1.0) for b in sb)


def test_non_finite_rows_leave_the_others(capsys):
    """NaN and infinity: nothing faults, every other row keeps its bytes."""
    d = dev()
    announce("non-finite rows")
    x = _draw(6, 512, F32, seed=2)
    bad = x.clone()
    bad[2, 5], bad[4, 500] = float("nan"), float("inf")
    fine = [0, 1, 3, 5]
    for kind in ("i8", "bf16", "fp8"):
        a = tp.tp_layernorm_rotate(x.to(d), out_kind=kind)
        b = tp.tp_layernorm_rotate(bad.to(d), out_kind=kind)
        a, b = (v if kind == "bf16" else v[0] for v in (a, b))
        assert torch.equal(a.view(torch.uint8)[fine], b.view(torch.uint8)[fine]), kind
    a, b = (tp.tp_quantize_fp8(v.to(d))[0].view(torch.uint8) for v in (x, bad))
    assert torch.equal(a[fine], b[fine])


# (a, c): rows a, a, c, 0 .. whose rotation has values c / 16 that fp32 rounds across
# the midpoint of two codes (they are subnormal there), under a normal scale
CROSSED = [("0x1.4510bep-113", "0x1.8abca4p-127"), ("0x1.0a7d3ep-113", "0x1.439b24p-127"), ("0x1.043b28p-113", "0x1.3c01a4p-127"),
           ("0x1.d0327ap-113", "0x1.19d82ep-126"), ("0x1.9b4c7cp-113", "0x1.f373ep-127"), ("0x1.8b2b02p-113", "0x1.dfdd5cp-127"),
           ("0x1.ef60e8p-113", "0x1.2cc6d2p-126"), ("0x1.00b378p-113", "0x1.37b854p-127")]


def test_rotated_values_beyond_fp32():
    """Rotated values are fp64: below fp32's normal numbers and above its largest
    they have codes like any others."""
    d = dev()
    announce("tp_quantize_fp8 rotated values beyond fp32")
    x = np.zeros((16, 256), dtype=np.float32)
    for i, (a, c) in enumerate(CROSSED):
        x[i, :3] = float.fromhex(a), float.fromhex(a), float.fromhex(c)
    rng = np.random.default_rng(4)
    x[8], x[9] = np.float32(3e38), rng.standard_normal(256) * 1e38
    x[10] = np.float32(-1e38)
    x[10, :128] *= np.float32(-2)
    x[11:] = (rng.standard_normal((5, 256)) * 1e-37).astype(np.float32)
    xt = torch.from_numpy(x)
    for rows in (xt, xt[:8], xt[8:11]):
        _check_quant(rows, rows.shape[0], 256, True, d, rows.to(d))


def test_layernorm_codes_beyond_fp32():
    """The same of normed rows under weights near the ends of fp32: rows of +-1
    are their own norm (eps far below)."""
    d = dev()
    announce("tp_layernorm_rotate weights at the ends of fp32")
    k = 512
    rng = np.random.default_rng(6)
    x = np.where(np.arange(k) % 2, 1.0, -1.0)[None, :].repeat(3, 0)
    x[1] = -x[1]
    x[2] = rng.standard_normal(k)
    for size in (1e38, 1e-37, 4e-36):
        gamma = np.minimum(size * (1 + np.abs(rng.standard_normal(k))), np.finfo(np.float32).max)
        gamma = torch.from_numpy(gamma.astype(np.float32))
        for rotate in (True, False):
            got = tp.tp_layernorm_rotate(torch.from_numpy(x.astype(np.float32)).to(d), gamma.to(d), eps=1e-30, rotate=rotate,
                                         out_kind="fp8")
            _check(x.astype(np.float32).astype(np.float64), gamma, None, 1e-30, rotate, "fp8", got)
