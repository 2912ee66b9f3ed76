"""Binding of the operators of a pre-norm block's branches: dropout, layer norm
and the products in 8-bit floating point.

    tp_dropout(x, drop_p, rng, residual)          -> drop(x) + residual (its own backward pass)
    tp_layernorm_rotate(x, gamma, beta, residual=, drop_p=, rng=)
                                                  -> codes, scales (or rows), and the new stream
    tp_layernorm_rotate_backward(dy, t, gamma)    -> dx, dbranch, dgamma, dbeta
    tp_quantize_fp8(x, block_rows, rotate, want)  -> e4m3 codes and a scale for each block of 128
    tp_qgemm_fp8(a, a_scales, b, b_scales)        -> C

Like the rest of the package, each function has the name of the C entry point
it calls, allocates what it is not given, and runs on the current stream of its
tensors' device (or on `stream`, whose allocations it then uses). All tensors
of a call sit on one device.
"""

import functools

import torch

from . import _lib
from ._lib import TP_A_PREROTATED, TP_A_ROTATE, TP_NORM_OUT_BF16, TP_NORM_OUT_FP8, TP_NORM_OUT_I8
from .block_ops import _device, _dt, _elsewhere, _empty, _mat, _raw_stream, _scratch, _vec, _weight

_F8 = torch.float8_e4m3fn
_KIND = {"i8": (TP_NORM_OUT_I8, torch.int8), "bf16": (TP_NORM_OUT_BF16, torch.bfloat16), "fp8": (TP_NORM_OUT_FP8, _F8)}
_BLOCK = 128  # elements that share a scale


@functools.lru_cache(maxsize=4096)
def _size_of(query, *sizes):
    """A workspace's size, which depends on the call's sizes alone (asked for
    anew it takes 0.5 us of a call of 8)."""
    return getattr(_lib.load(), query)(*sizes)


def _up(v):
    return -(-v // _BLOCK) * _BLOCK


def _rng_ptr(rng, drop_p):
    """Pointer of a dropout's seed and offset (None where nothing can drop)."""
    if rng is None:
        if drop_p != 0:
            raise ValueError("a dropout needs rng, an int64 tensor of seed and offset")
        return None
    return _vec(rng, "rng", 2, torch.int64).data_ptr()


def _out(t, name, rows, cols, dtype, device):
    """A given output checked, or a new one; and its row pitch."""
    if t is None:
        return _empty((rows, cols), (cols, 1), dtype=dtype, device=device), cols
    return t, _mat(t, name, rows, cols, dtype)


def tp_dropout(x, drop_p, rng=None, residual=None, out_dtype=None, out=None, stream=None):
    """drop(x) + residual: x / (1 - drop_p) where the element is kept, 0 where
    not. rng: int64 tensor of two, seed and offset, read on the device when the
    call runs; the same rng, width and drop_p give the same mask, so the call on
    a gradient (without residual) is the backward pass. Default dtype of the
    result: the residual's, else x's. out may be x or residual itself."""
    index = _device(x, "rng residual out", (rng, residual, out))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_dropout(x, drop_p, rng, residual, out_dtype, out)
    ldx = _mat(x, "x")
    m, k = x.shape
    rng_ptr = _rng_ptr(rng, drop_p)
    if out is None:
        dtype = out_dtype or (x if residual is None else residual).dtype
        per = 8 if dtype == torch.bfloat16 else 4  # rows start at multiples of 16 bytes
        ldy = -(-k // per) * per
        out = _empty((m, k), (ldy, 1), dtype=dtype, device=x.device)
    else:
        ldy = _mat(out, "out", m, k, out_dtype)
    r_ptr, ldr = None, 0
    if residual is not None:
        r_ptr, ldr = residual.data_ptr(), _mat(residual, "residual", m, k, out.dtype)
    _lib.check(_lib.load().tp_dropout(x.data_ptr(), _dt(x, "x"), ldx, r_ptr, ldr, drop_p, rng_ptr, m, k,
                                      out.data_ptr(), _dt(out, "out"), ldy, _raw_stream(index)))
    return out


def tp_layernorm_rotate(x, gamma=None, beta=None, eps=1e-5, residual=None, drop_p=0.0, rng=None, rotate=True,
                        out_kind="i8", out=None, scales=None, sum_out=None, stream=None):
    """t = drop(x) + residual (fp32, rounded to the residual's dtype) or x; the
    layer norm of t's rows, times gamma plus beta, rotated per 256-group (unless
    rotate=False), as int8 codes with one fp32 scale per row (out_kind "i8"), as
    bf16 rows ("bf16") or as e4m3 codes with scales [k / 128, m] ("fp8").
    Returns (codes, scales) or rows; with a residual also t, the new stream.
    drop_p and rng as in tp_dropout (a dropout needs a residual). sum_out may be
    residual (or x) itself."""
    index = _device(x, "gamma beta residual rng out scales sum_out", (gamma, beta, residual, rng, out, scales, sum_out))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_layernorm_rotate(x, gamma, beta, eps, residual, drop_p, rng, rotate, out_kind, out, scales,
                                       sum_out)
    if out_kind not in _KIND:
        raise ValueError("out_kind must be 'i8', 'bf16' or 'fp8'")
    kind, y_dtype = _KIND[out_kind]
    ldx = _mat(x, "x")
    m, k = x.shape
    device = x.device
    g_ptr, g_dt = _weight(gamma, "gamma", k)
    b_ptr, b_dt = _weight(beta, "beta", k)
    if gamma is not None and beta is not None and g_dt != b_dt:
        raise TypeError("gamma and beta must have one dtype")
    rng_ptr = _rng_ptr(rng, drop_p)
    r_ptr = s_ptr = sc_ptr = None
    ldr = lds = s_dt = ldsc = 0
    if residual is not None:
        ldr = _mat(residual, "residual", m, k)
        s_dt = _dt(residual, "residual")
        sum_out, lds = _out(sum_out, "sum_out", m, k, residual.dtype, device)
        r_ptr, s_ptr = residual.data_ptr(), sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    out, ldy = _out(out, "out", m, k, y_dtype, device)
    if kind == TP_NORM_OUT_I8:
        if scales is None:
            scales = _empty((m,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(scales, "scales", m, torch.float32)
        sc_ptr = scales.data_ptr()
    elif kind == TP_NORM_OUT_FP8:
        scales, ldsc = _out(scales, "scales", k // _BLOCK, m, torch.float32, device)
        sc_ptr = scales.data_ptr()
    elif scales is not None:
        raise ValueError("scales belong to out_kind 'i8' and 'fp8'")
    _lib.check(_lib.load().tp_layernorm_rotate(
        x.data_ptr(), _dt(x, "x"), ldx, r_ptr, ldr, s_ptr, lds, s_dt, g_ptr, b_ptr, g_dt if gamma is not None else b_dt,
        eps, drop_p, rng_ptr, TP_A_ROTATE if rotate else TP_A_PREROTATED, m, k, kind, out.data_ptr(), ldy, sc_ptr, ldsc,
        _raw_stream(index)))
    got = (out,) if kind == TP_NORM_OUT_BF16 else (out, scales)
    if residual is not None:
        got += (sum_out,)
    return got if len(got) > 1 else out


def tp_layernorm_backward_workspace_size(m, k):
    """Bytes of workspace tp_layernorm_rotate_backward needs for dgamma and dbeta."""
    return _size_of("tp_layernorm_backward_workspace_size", m, k)


def tp_layernorm_rotate_backward(dy, t, gamma=None, eps=1e-5, dsum=None, drop_p=0.0, rng=None, rotate=True,
                                 dx_dtype=None, want_dgamma=True, want_dbeta=True, dx=None, dbranch=None, dgamma=None,
                                 dbeta=None, workspace=None, stream=None):
    """Gradients of tp_layernorm_rotate (quantization straight through): dy is
    the gradient of its rows (rotated ones unless rotate=False), t its sum (or
    x), dsum the gradient that reaches the stream from behind, drop_p and rng the
    forward's. Returns (dx, dbranch, dgamma, dbeta): the residual's gradient,
    x's (drop(dx); None where drop_p is 0: it is dx), and the weights' (None
    where they are not wanted). dx (default dtype: dsum's, else t's) may be dsum
    itself, or dy itself where neither weight's gradient is wanted."""
    index = _device(dy, "t gamma dsum rng dx dbranch dgamma dbeta workspace",
                    (t, gamma, dsum, rng, dx, dbranch, dgamma, dbeta, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_layernorm_rotate_backward(dy, t, gamma, eps, dsum, drop_p, rng, rotate, dx_dtype, want_dgamma,
                                                want_dbeta, dx, dbranch, dgamma, dbeta, workspace)
    lddy = _mat(dy, "dy")
    m, k = dy.shape
    device = dy.device
    ldt = _mat(t, "t", m, k)
    g_ptr, g_dt = _weight(gamma, "gamma", k)
    rng_ptr = _rng_ptr(rng, drop_p)
    if dx is None:
        dx_dtype = dx_dtype or (t if dsum is None else dsum).dtype
    dx, lddx = _out(dx, "dx", m, k, dx_dtype, device)
    ds_ptr, ldds = None, 0
    if dsum is not None:
        ds_ptr, ldds = dsum.data_ptr(), _mat(dsum, "dsum", m, k, dx.dtype)
    b_ptr, lddb = None, 0
    if drop_p != 0 or dbranch is not None:
        dbranch, lddb = _out(dbranch, "dbranch", m, k, dx.dtype, device)
        b_ptr = dbranch.data_ptr()
    dg_ptr = db_ptr = ws_ptr = ws = None
    ws_bytes = 0
    if want_dgamma or dgamma is not None:
        if dgamma is None:
            dgamma = _empty((k,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(dgamma, "dgamma", k, torch.float32)
        dg_ptr = dgamma.data_ptr()
    if want_dbeta or dbeta is not None:
        if dbeta is None:
            dbeta = _empty((k,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(dbeta, "dbeta", k, torch.float32)
        db_ptr = dbeta.data_ptr()
    if dg_ptr is not None or db_ptr is not None:
        ws_ptr, ws_bytes, ws = _scratch(workspace, tp_layernorm_backward_workspace_size(m, k), device)
    _lib.check(_lib.load().tp_layernorm_rotate_backward(
        dy.data_ptr(), _dt(dy, "dy"), lddy, TP_A_ROTATE if rotate else TP_A_PREROTATED, t.data_ptr(), _dt(t, "t"),
        ldt, g_ptr, g_dt, eps, ds_ptr, ldds, drop_p, rng_ptr, m, k, dx.data_ptr(), _dt(dx, "dx"), lddx, b_ptr, lddb,
        dg_ptr, db_ptr, ws_ptr, ws_bytes, _raw_stream(index)))
    return dx, dbranch, dgamma, dbeta


def tp_quantize_fp8(x, block_rows=1, rotate=False, want="rows", q=None, scales=None, qt=None, scales_t=None,
                    stream=None):
    """e4m3 codes of x [m, k] (of its rotation with rotate=True) with an fp32
    scale for each block of 128. want "rows": (codes [m, kp], scales [kp / 128,
    m]), kp being k rounded up to 128, for a product over k; "cols": (codes of
    the transpose [k, mp], scales [mp / 128, k]), for a product over m; "both":
    all four. With block_rows=128 a scale covers 128 x 128 elements (weights):
    scales [mp / 128, kp / 128], and the same codes transposed with scales
    [kp / 128, mp / 128]."""
    index = _device(x, "q scales qt scales_t", (q, scales, qt, scales_t))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_quantize_fp8(x, block_rows, rotate, want, q, scales, qt, scales_t)
    if want not in ("rows", "cols", "both"):
        raise ValueError("want must be 'rows', 'cols' or 'both'")
    ldx = _mat(x, "x")
    m, k = x.shape
    mp, kp, device = _up(m), _up(k), x.device
    blocks = block_rows == _BLOCK
    q_ptr = s_ptr = qt_ptr = st_ptr = None
    ldq = lds = ldqt = ldst = 0
    if want != "cols":
        q, ldq = _out(q, "q", m, kp, _F8, device)
        rows, cols = (mp // _BLOCK, kp // _BLOCK) if blocks else (kp // _BLOCK, m)
        scales, lds = _out(scales, "scales", rows, cols, torch.float32, device)
        q_ptr, s_ptr = q.data_ptr(), scales.data_ptr()
    elif q is not None or scales is not None:
        raise ValueError("q and scales belong to want 'rows' and 'both'")
    if want != "rows":
        qt, ldqt = _out(qt, "qt", k, mp, _F8, device)
        rows, cols = (kp // _BLOCK, mp // _BLOCK) if blocks else (mp // _BLOCK, k)
        scales_t, ldst = _out(scales_t, "scales_t", rows, cols, torch.float32, device)
        qt_ptr, st_ptr = qt.data_ptr(), scales_t.data_ptr()
    elif qt is not None or scales_t is not None:
        raise ValueError("qt and scales_t belong to want 'cols' and 'both'")
    if m > 0 and k > 0:
        _lib.check(_lib.load().tp_quantize_fp8(
            x.data_ptr(), _dt(x, "x"), ldx, m, k, TP_A_ROTATE if rotate else TP_A_PREROTATED, block_rows, q_ptr, ldq,
            s_ptr, lds, qt_ptr, ldqt, st_ptr, ldst, _raw_stream(index)))
    if want == "both":
        return q, scales, qt, scales_t
    return (q, scales) if want == "rows" else (qt, scales_t)


def tp_qgemm_fp8_workspace_size(m, n, k, out_dtype=torch.float32):
    """Bytes of workspace tp_qgemm_fp8 needs (0: none)."""
    return _size_of("tp_qgemm_fp8_workspace_size", m, n, k, _lib.TP_BF16 if out_dtype == torch.bfloat16 else _lib.TP_F32)


def tp_qgemm_fp8(a, a_scales, b, b_scales, b_block_rows=128, out_dtype=torch.float32, out=None, workspace=None,
                 stream=None):
    """C [m, n] = a . b^T of e4m3 codes [m, k] and [n, k] with a scale for each
    block of 128 along k: a_scales [k / 128, m]; b_scales [n / 128 rounded up,
    k / 128] (a scale for 128 x 128 codes), or with b_block_rows=1 [k / 128, n].
    A new C has rows at multiples of 16 bytes, as the other operators take them.
    k == 0 (the weight's gradient of no tokens) gives zeros."""
    index = _device(a, "a_scales b b_scales out workspace", (a_scales, b, b_scales, out, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_qgemm_fp8(a, a_scales, b, b_scales, b_block_rows, out_dtype, out, workspace)
    lda = _mat(a, "a", dtype=_F8)
    m, k = a.shape
    ldb = _mat(b, "b", cols=k, dtype=_F8)
    n, kb = b.shape[0], k // _BLOCK
    ldsa = _mat(a_scales, "a_scales", kb, m, torch.float32)
    rows, cols = (kb, n) if b_block_rows == 1 else (_up(n) // _BLOCK, kb)
    ldsb = _mat(b_scales, "b_scales", rows, cols, torch.float32)
    if out is None:
        per = 8 if out_dtype == torch.bfloat16 else 4
        ldc = -(-n // per) * per
        out = _empty((m, n), (ldc, 1), dtype=out_dtype, device=a.device)
    else:
        ldc = _mat(out, "out", m, n)
    out_dt = _dt(out, "out")
    if k == 0 and b_block_rows in (1, _BLOCK):  # no tokens: the C entry point has no products of nothing
        return out.zero_()
    need = tp_qgemm_fp8_workspace_size(m, n, k, out.dtype)
    ws_ptr, ws_bytes, ws = (None, 0, None) if workspace is None and not need else _scratch(workspace, need, a.device)
    _lib.check(_lib.load().tp_qgemm_fp8(
        a.data_ptr(), lda, a_scales.data_ptr(), ldsa, b.data_ptr(), ldb, b_scales.data_ptr(), ldsb, b_block_rows, m, n,
        k, out.data_ptr(), out_dt, ldc, ws_ptr, ws_bytes, _raw_stream(index)))
    return out
