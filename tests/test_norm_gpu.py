"""tp_rmsnorm_rotate and its gradients against the fp64 oracle.

* codes and scales equal to the oracle's: both sides decide in 64 bits, and
  differ only where a quotient is within about 1e-13 of a tie (or the scale of
  a midpoint of fp32), which random rows of these sizes do not reach;
* the new stream bit for bit;
* bf16 rows and gradients inside the bounds of the fp32 arithmetic.
"""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64, host

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# one group to 64, rows that share a block (fewer than four groups) and rows
# that take one, ragged against 16 sets, four waves and sixteen
SHAPES = [(1, 256), (37, 256), (5, 512), (16, 768), (3, 1024), (130, 1280), (7, 3072), (2, 4096), (3, 4352),
          (2, 12288), (1, 16384)]


def _draw(m, k, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float32) * np.float32(scale)
    x[:, rng.choice(k, size=max(1, k // 200), replace=False)] *= np.float32(30.0)
    return torch.from_numpy(x).to(dtype)


def _gamma(k, dtype, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((1.0 + 0.1 * rng.standard_normal(k)).astype(np.float32)).to(dtype)


def _check(t64, gamma, eps, rotate, kind, got):
    g = None if gamma is None else f64(gamma)
    h = oracle.rmsnorm(t64, g, eps)
    if kind == "i8":
        q, s = oracle.quantize_activations_int8(h, rotate=rotate)
        assert np.array_equal(host(got[1]), s), f"{int(np.sum(host(got[1]) != s))} scales differ"
        assert np.array_equal(host(got[0]), q), f"{int(np.sum(host(got[0]) != q))} codes differ"
    else:
        y, bound = B.norm_rows(t64, g, eps, rotate)
        B.assert_close(f64(got[0]), y, bound, True, "rows")


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("xdt,sdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, None), (BF16, None), (F32, F32)])
def test_norm_shapes_and_types(m, k, xdt, sdt):
    d = dev()
    announce("tp_rmsnorm_rotate", m, k, xdt, sdt)
    x = _draw(m, k, xdt, seed=m + k)
    gamma = _gamma(k, BF16 if m % 2 else F32, seed=k)
    res = None if sdt is None else _draw(m, k, sdt, seed=m + k + 1, scale=2.0)
    t64 = f64(x) if res is None else oracle.stream_sum(f64(x), f64(res), sdt == BF16)
    for kind in ("i8", "bf16"):
        for rotate in (True, False):
            got = tp.tp_rmsnorm_rotate(x.to(d), gamma.to(d), eps=1e-6, residual=None if res is None else res.to(d),
                                       rotate=rotate, out_kind=kind)
            got = got if isinstance(got, tuple) else (got,)
            if res is not None:
                assert got[-1].dtype == sdt and np.array_equal(f64(got[-1]), t64), "the new stream differs"
            _check(t64, gamma, 1e-6, rotate, kind, got)


@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_norm_without_weight_and_special_rows(kind):
    """No gamma; rows of zeros, rows far below eps, a single element, huge
    values, and a row whose scale is subnormal."""
    d = dev()
    announce("tp_rmsnorm_rotate special rows", kind)
    rng = np.random.default_rng(8)
    x = rng.standard_normal((7, 512)).astype(np.float32)
    x[1] = 0.0
    x[2] *= np.float32(1e-20)
    x[3] = 0.0
    x[3, 300] = -3.0
    x[4] *= np.float32(1e18)
    x[5] *= np.float32(1e-39)
    xt = torch.from_numpy(x)
    for eps in (1e-6, 1e-30):
        got = tp.tp_rmsnorm_rotate(xt.to(d), None, eps=eps, out_kind=kind)
        if kind == "bf16":
            got = (got,)
        _check(f64(xt), None, eps, True, kind, got)
        assert np.all(host(got[0].float())[1] == 0)


def test_norm_in_place_stream_and_padded_views():
    d = dev()
    announce("tp_rmsnorm_rotate in place, padded views")
    m, k = 21, 1024
    x = _draw(m, k, F32, seed=1)
    res = _draw(m, k, F32, seed=2)
    gamma = _gamma(k, F32, seed=3)
    t64 = oracle.stream_sum(f64(x), f64(res), False)
    xb = torch.full((m, k + 128), 5.0, device=d)
    xb[:, 64:64 + k] = x.to(d)
    stream = torch.full((m + 2, k + 8), 9.0, device=d)
    stream[1:-1, :k] = res.to(d)
    qb = torch.full((m + 2, k + 64), 7, dtype=torch.int8, device=d)
    sb = torch.full((m + 8,), -1.0, device=d)
    view = stream[1:-1, :k]
    q, s, t = tp.tp_rmsnorm_rotate(xb[:, 64:64 + k], gamma.to(d), residual=view, out=qb[1:-1, 32:32 + k],
                                   scales=sb[4:4 + m], sum_out=view)
    assert t is view and np.array_equal(f64(view), t64)
    _check(t64, gamma, 1e-6, True, "i8", (q, s))
    assert torch.all(stream[0] == 9) and torch.all(stream[-1] == 9) and torch.all(stream[:, k:] == 9)
    assert torch.all(qb[0] == 7) and torch.all(qb[-1] == 7) and torch.all(qb[:, :32] == 7)
    assert torch.all(qb[:, 32 + k:] == 7) and torch.all(sb[:4] == -1) and torch.all(sb[4 + m:] == -1)
    # the stream written over x
    xd = x.to(d)
    rows, t = tp.tp_rmsnorm_rotate(xd, gamma.to(d), residual=res.to(d), sum_out=xd, out_kind="bf16")
    assert t is xd and np.array_equal(f64(xd), t64)
    _check(t64, gamma, 1e-6, True, "bf16", (rows,))


def test_norm_rows_with_nan_or_infinity_leave_the_others():
    d = dev()
    announce("tp_rmsnorm_rotate non-finite rows")
    for k in (512, 2048):
        x = _draw(40, k, F32, seed=k)
        clean = [host(v) for v in tp.tp_rmsnorm_rotate(x.to(d), None)]
        bad = x.clone()
        bad[3, 7], bad[17, 100], bad[18, 200] = float("nan"), float("inf"), float("-inf")
        q, s = (host(v) for v in tp.tp_rmsnorm_rotate(bad.to(d), None))
        keep = np.setdiff1d(np.arange(40), [3, 17, 18])
        assert np.array_equal(q[keep], clean[0][keep]) and np.array_equal(s[keep], clean[1][keep])
        assert q.min() >= -127


def test_norm_many_rows_walked_by_few_blocks():
    """More rows than blocks: every row once, whatever block walks it."""
    d = dev()
    announce("tp_rmsnorm_rotate many rows")
    for m, k in ((40000, 256), (5000, 1024)):
        g = torch.Generator(device=d)
        g.manual_seed(m)
        x = torch.randn((m, k), device=d, generator=g)
        q, s = tp.tp_rmsnorm_rotate(x, None)
        sel = np.unique(np.concatenate([np.arange(40), np.arange(m - 40, m), np.arange(0, m, 97)]))
        sel_t = torch.from_numpy(sel).to(d)
        _check(f64(x[sel_t]), None, 1e-6, True, "i8", (q[sel_t], s[sel_t]))


@pytest.mark.parametrize("m,k", SHAPES + [(700, 512), (1100, 1024)])
@pytest.mark.parametrize("gdt,tdt,xdt", [(F32, BF16, BF16), (BF16, F32, F32), (F32, F32, F32), (BF16, BF16, F32),
                                         (BF16, BF16, BF16)])
def test_norm_backward(m, k, gdt, tdt, xdt):
    d = dev()
    announce("tp_rmsnorm_rotate_backward", m, k, gdt, tdt, xdt)
    dy = _draw(m, k, gdt, seed=m + k, scale=0.02)
    t = _draw(m, k, tdt, seed=m + k + 1)
    ds = _draw(m, k, xdt, seed=m + k + 2, scale=0.02)
    gamma = _gamma(k, F32 if m % 2 else BF16, seed=k)
    for rotate, dsum, gam in ((True, ds, gamma), (False, None, gamma), (True, None, None)):
        dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None if gam is None else gam.to(d), eps=1e-6,
                                               dsum=None if dsum is None else dsum.to(d), rotate=rotate, dx_dtype=xdt)
        adds = m + 64  # rows one after the other, then the blocks' sums
        want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), None if gam is None else f64(gam), 1e-6,
                                                None if dsum is None else f64(dsum), rotate, adds)
        B.assert_close(f64(dx), want, bound, xdt == BF16, "dx")
        B.assert_close(f64(dg), wdg, bdg, False, "dgamma")


def test_norm_backward_in_place_unwanted_and_empty():
    d = dev()
    announce("tp_rmsnorm_rotate_backward in place")
    m, k = 33, 768
    dy, t, ds = (_draw(m, k, F32, seed=s) for s in (1, 2, 3))
    gamma = _gamma(k, F32, seed=4).to(d)
    want, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), gamma, dsum=ds.to(d))
    buf = ds.to(d)
    dx, none = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), gamma, dsum=buf, dx=buf, want_dgamma=False)
    assert none is None and dx is buf and torch.equal(dx, want)
    buf = dy.to(d)
    dx, dg2 = tp.tp_rmsnorm_rotate_backward(buf, t.to(d), gamma, dsum=ds.to(d), dx=buf)
    assert torch.equal(dx, want) and torch.equal(dg, dg2)
    empty = torch.empty((0, k), device=d)
    dx, dg = tp.tp_rmsnorm_rotate_backward(empty, empty, gamma)
    assert dx.shape == (0, k) and torch.all(dg == 0)
    q, s = tp.tp_rmsnorm_rotate(empty, gamma)
    assert q.shape == (0, k) and s.shape == (0,)


@pytest.mark.parametrize("m,k", [(9001, 256), (2700, 768), (2101, 1024)])
def test_norm_backward_short_rows_share_blocks(m, k):
    """More rows than all blocks take at a time, several of them a block."""
    d = dev()
    announce("tp_rmsnorm_rotate_backward short rows", m, k)
    dy, t, ds = _draw(m, k, F32, seed=m, scale=0.02), _draw(m, k, BF16, seed=m + 1), _draw(m, k, BF16, seed=m + 2)
    gamma = _gamma(k, F32, seed=k)
    dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), gamma.to(d), dsum=ds.to(d))
    want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), f64(gamma), 1e-6, f64(ds), True, m + 64)
    B.assert_close(f64(dx), want, bound, True, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")


@pytest.mark.parametrize("m,k", [(40, 512), (600, 256), (30, 2048), (6, 8192)])
def test_norm_backward_special_rows(m, k):
    """Rows of zeros at the smallest eps, and non-finite rows beside others:
    their gradients are their own."""
    d = dev()
    announce("tp_rmsnorm_rotate_backward special rows", m, k)
    dy, t = _draw(m, k, F32, seed=m, scale=0.02), _draw(m, k, F32, seed=m + 1)
    t[2] = 0.0
    for eps in (1e-6, 1e-30):
        dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None, eps=eps)
        want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), None, eps, None, True, m + 64)
        B.assert_close(f64(dx), want, bound, False, "dx")
        B.assert_close(f64(dg), wdg, bdg, False, "dgamma")
    t[1, 7], t[4, 100], dy[5, 200] = float("nan"), float("inf"), float("-inf")
    bad, _ = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None, eps=1e-30)
    keep = [i for i in range(m) if i not in (1, 4, 5)]
    assert torch.equal(bad[keep], dx[keep])
