"""Forms of the operators around the projections that the tests of each operator
leave out, against the fp64 oracle: few rows at every padded rank (the waves of a block share a
chunk), several tokens a block with a ragged last batch, blocks that walk rows
or tokens beyond the largest grid, and wide rows of which a block takes several.
"""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64, host
from tests.test_rope_gpu import _draw as _rope_draw, _gamma as _rope_gamma, _plan
from tests.test_side_gpu import _codes, _mat, _on, _parts

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------------ side path
def _check_down(m, k, r, adt):
    d = dev()
    announce("tp_lora_down_prequantized", m, k, r, adt)
    qa, sa = _codes(m, k, seed=m + k + r)
    a = _mat((r, k), adt, seed=r, scale=k ** -0.5)
    t = host(tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), _on(d, a, k))).astype(np.float64)
    x, a64 = f64(qa) * f64(sa)[:, None], f64(a[:, :k])
    B.assert_sum(t[:, :r], oracle.lora_down_codes(qa.numpy(), sa.numpy(), a64), np.abs(x) @ np.abs(a64).T,
                 k * _parts(adt) + 32, "T")
    assert np.all(t[:, r:] == 0)


@pytest.mark.parametrize("m", [1, 7, 16])
@pytest.mark.parametrize("k,r", [(256, 32), (1280, 24), (4096, 33), (12288, 64), (768, 17)])
@pytest.mark.parametrize("adt", [BF16, F32])
def test_down_few_rows_every_rank(m, k, r, adt):
    _check_down(m, k, r, adt)


@pytest.mark.parametrize("m", [17, 40, 64, 65])
@pytest.mark.parametrize("k,r", [(512, 8), (1280, 16), (1280, 32), (768, 40), (3840, 64)])
@pytest.mark.parametrize("adt", [BF16, F32])
def test_down_one_and_two_row_tiles_every_rank(m, k, r, adt):
    _check_down(m, k, r, adt)


@pytest.mark.parametrize("m,n,k,r", [(1, 300, 512, 32), (1, 1160, 256, 64), (5, 1160, 512, 33), (7, 2052, 256, 24),
                                     (16, 520, 256, 64), (16, 4100, 768, 32), (12, 40, 256, 17)])
@pytest.mark.parametrize("ydt,bdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_grad_few_rows_every_rank(m, n, k, r, ydt, bdt):
    d = dev()
    announce("tp_lora_grad_prequantized", m, n, k, r, ydt, bdt)
    alpha, rotate = 0.75, bool(m % 2)
    qa, sa = _codes(m, k, seed=m + k)
    dy, b = _mat((m, n), ydt, seed=n, scale=0.02), _mat((n, r), bdt, seed=n + 1)
    t = torch.full((m, 64), 3.0)
    t[:, :r] = _mat((m, r), F32, seed=n + 2)[:, :r]
    got = tp.tp_lora_grad_prequantized(_on(d, dy, n), qa.to(d), sa.to(d), t.to(d), _on(d, b, r), alpha, rotate=rotate)
    da, db, dt = (host(v).astype(np.float64) for v in got)
    y64, b64, t64 = f64(dy[:, :n]), f64(b[:, :r]), f64(t[:, :r])
    wda, wdb, wdt = oracle.lora_grad_codes(y64, qa.numpy(), sa.numpy(), t64, b64, alpha, rotate=rotate)
    mag_dt = alpha * np.abs(y64) @ np.abs(b64)
    terms = n * _parts(ydt, bdt) + 64
    B.assert_sum(dt[:, :r], wdt, mag_dt, terms, "dT")
    assert np.all(dt[:, r:] == 0)
    B.assert_sum(db, wdb, alpha * np.abs(y64).T @ np.abs(t64), m * _parts(ydt, F32) + 64, "dB")
    mag_da = mag_dt.T @ np.abs(f64(qa) * f64(sa)[:, None])
    if rotate:
        mag_da = B.group_l1(mag_da) / 16.0
    B.assert_sum(da, wda, mag_da, terms + 4 + 3 * m + 64 + (8 if rotate else 0), "dA")


# ------------------------------------------------------------------------ rope
# two tokens a block (by their number), four with three in the last batch, two by
# the width of the rotation, four tokens without a rotation, and more batches
# than the grid has blocks
BATCHES = [(2049, 2, 1, 16, 8, 2), (4099, 3, 1, 24, 8, 3), (4101, 1, 1, 256, 128, 2), (4102, 5, 0, 32, 12, 1),
           (4097, 2, 2, 16, 0, 1), (33001, 1, 1, 8, 4, 1)]


@pytest.mark.parametrize("m,hq,hk,d,pairs,axes", BATCHES)
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("xdt,odt", [(F32, F32), (BF16, BF16)])
def test_rope_of_several_tokens_a_block(m, hq, hk, d, pairs, axes, layout, xdt, odt):
    dv = dev()
    announce("tp_qk_norm_rope batches", m, hq, hk, d, pairs, axes, layout, xdt)
    w, c = (hq + hk) * d, hq * d
    qk, dy = _rope_draw((m, w), xdt, m + d, 1.5), _rope_draw((m, w), odt, m + d + 1, 0.02)
    pos, freq, axis = _plan(m, pairs, axes, seed=d, far=5000)
    qkd, dyd = qk.to(dv), dy.to(dv)
    how = (d, pos.to(dv), freq.to(dv) if pairs else None, axis, layout)
    halves = layout == "halves"
    # terms a column of dgamma goes through: a lane's tokens and heads, a
    # block's groups of lanes, the blocks in 16 slices
    adds = m * max(hq, hk) // 1024 + 256 + 64 + 16 + 64
    for qg, kg in ((None, None), (_rope_gamma(d, BF16, 1), _rope_gamma(d, BF16, 2))):
        on = [None if g is None else g.to(dv) for g in (qg, kg)]
        out = tp.tp_qk_norm_rope(qkd[:, :c], qkd[:, c:], *how, *on, eps=1e-5, out_dtype=odt)
        grads = tp.tp_qk_norm_rope_backward(dyd[:, :c], dyd[:, c:], qkd[:, :c], qkd[:, c:], *how, *on, eps=1e-5,
                                            dx_dtype=odt)
        for lo, hi, gamma, i in ((0, c, qg, 0), (c, w, kg, 1)):
            if lo == hi:
                continue
            g64 = None if gamma is None else f64(gamma)
            plan = (d, pos.numpy(), freq.numpy(), axis, halves, g64, 1e-5)
            want, bound = B.rope_forward(f64(qk[:, lo:hi]), *plan)
            B.assert_close(f64(out[i]), want, bound, odt == BF16, "out")
            want, bound, wdg, bdg = B.rope_backward(f64(dy[:, lo:hi]), f64(qk[:, lo:hi]), *plan, adds)
            B.assert_close(f64(grads[i]), want, bound, odt == BF16, "dx")
            if gamma is not None:
                B.assert_close(f64(grads[2 + i]), wdg, bdg, False, "dgamma")


# ------------------------------------------------------------------------ norm
@pytest.mark.parametrize("m,k,rows", [(65536 * 16 + 37, 256, 16), (65536 * 5 + 3, 768, 5), (65536 + 9, 1024, 1)])
@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_norm_blocks_walk_rows(m, k, rows, kind):
    """More rows than 65536 blocks hold at a time: the first rows, those around
    the end of the first sweep and the last ones, and the blocks' second row."""
    d = dev()
    announce("tp_rmsnorm_rotate walking blocks", m, k, kind)
    g = torch.Generator(device=d).manual_seed(k)
    x = torch.empty((m, k), dtype=BF16, device=d).normal_(generator=g)
    res = torch.empty((m, k), dtype=BF16, device=d).normal_(generator=g)
    got = tp.tp_rmsnorm_rotate(x, None, residual=res, out_kind=kind)
    sweep = 65536 * rows
    sel = np.unique(np.concatenate([np.arange(40), np.arange(sweep - 40, m), np.arange(0, m, 9973)]))
    sel_t = torch.from_numpy(sel).to(d)
    t64 = oracle.stream_sum(f64(x[sel_t]), f64(res[sel_t]), True)
    assert np.array_equal(f64(got[-1][sel_t]), t64)
    if kind == "i8":
        q, s = oracle.quantize_activations_int8(oracle.rmsnorm(t64, None, 1e-6))
        assert np.array_equal(host(got[1][sel_t]), s) and np.array_equal(host(got[0][sel_t]), q)
    else:
        want, bound = B.norm_rows(t64, None, 1e-6, True)
        B.assert_close(f64(got[0][sel_t]), want, bound, True, "rows")


@pytest.mark.parametrize("m,k", [(700, 4352), (1100, 8192), (520, 16384), (513, 12288)])
@pytest.mark.parametrize("gdt,tdt,xdt,with_dsum", [(F32, BF16, BF16, True), (F32, F32, F32, True),
                                                   (BF16, BF16, F32, False)])
def test_norm_backward_of_many_wide_rows(m, k, gdt, tdt, xdt, with_dsum):
    """Rows of more than 16 groups, more of them than blocks: a block takes
    several and keeps their part of dgamma."""
    d = dev()
    announce("tp_rmsnorm_rotate_backward wide rows", m, k, gdt, tdt, xdt)
    rng = np.random.default_rng(m)
    draw = lambda s: torch.from_numpy(rng.standard_normal((m, k), dtype=np.float32) * np.float32(s))  # noqa: E731
    dy, t = draw(0.02).to(gdt), draw(1.0).to(tdt)
    ds = draw(0.02).to(xdt) if with_dsum else None
    gamma = torch.from_numpy((1.0 + 0.1 * rng.standard_normal(k)).astype(np.float32))
    dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), gamma.to(d), dsum=None if ds is None else ds.to(d),
                                           dx_dtype=xdt)
    want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), f64(gamma), 1e-6, None if ds is None else f64(ds), True,
                                            m + 64)
    B.assert_close(f64(dx), want, bound, xdt == BF16, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")


@pytest.mark.parametrize("m,k", [(3, 4352), (512, 8192), (300, 12288), (40, 16384)])
@pytest.mark.parametrize("gdt,tdt,xdt", [(F32, BF16, BF16), (F32, F32, F32), (BF16, BF16, F32), (BF16, F32, BF16)])
def test_norm_backward_of_a_wide_row_a_block_with_a_stream_gradient(m, k, gdt, tdt, xdt):
    d = dev()
    announce("tp_rmsnorm_rotate_backward a wide row a block", m, k, gdt, tdt, xdt)
    rng = np.random.default_rng(m + k)
    draw = lambda s: torch.from_numpy(rng.standard_normal((m, k), dtype=np.float32) * np.float32(s))  # noqa: E731
    dy, t, ds = draw(0.02).to(gdt), draw(1.0).to(tdt), draw(0.02).to(xdt)
    dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None, dsum=ds.to(d))
    want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), None, 1e-6, f64(ds), True, m + 64)
    B.assert_close(f64(dx), want, bound, xdt == BF16, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")
