"""Binding of the operators around the projections of a transformer block.

    tp_rmsnorm_rotate(x, gamma, residual)         -> codes, scales (or rows), and the new stream
    tp_rmsnorm_rotate_backward(dy, t, gamma)      -> dx, dgamma
    tp_lora_down_prequantized(qa, sa, lora_a)     -> T
    tp_lora_grad_prequantized(dy, qa, sa, t, lora_b, alpha)
                                                  -> dA, dB, dT
    tp_qk_norm_rope(q, k, head_dim, positions, inv_freq)          -> q, k turned to their positions
    tp_qk_norm_rope_backward(dq_out, dk_out, q, k, head_dim, ...) -> dq, dk, dq_gamma, dk_gamma

Like the rest of the package, each function has the name of the C entry point
it calls, allocates what it is not given, and runs on the current stream of its
tensors' device (or on `stream`, whose allocations it then uses). All tensors
of a call sit on one device.
"""

import torch

from . import _lib
from ._lib import (TP_A_PREROTATED, TP_A_ROTATE, TP_NORM_OUT_BF16, TP_NORM_OUT_I8, TP_ROPE_HALVES,
                   TP_ROPE_INTERLEAVED)

_DTYPE = {torch.float32: _lib.TP_F32, torch.bfloat16: _lib.TP_BF16}
_KIND = {"i8": (TP_NORM_OUT_I8, torch.int8), "bf16": (TP_NORM_OUT_BF16, torch.bfloat16)}


# A call on a handful of rows takes less time on the GPU than in Python (a
# single token's rope: 4 us against 10), so the checks below take the short way
# where everything is in order, and what a call allocates itself is not checked.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_empty = torch.empty_strided


def _dt(t, name):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _device(first, names, others):
    """The index of the one CUDA (HIP) device of a call's tensors (None: not
    given); names are the others', for the message."""
    try:
        index = first.get_device()
        for t in others:
            if t is not None and t.get_device() != index:
                index = -1
    except AttributeError:
        index = -1
    if index < 0:
        _device_error(first, names.split(), others)
    return index


def _device_error(first, names, others):
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("the operands must be CUDA (HIP) tensors")
    for name, t in zip(names, others):
        if t is not None and (not isinstance(t, torch.Tensor) or t.device != first.device):
            raise ValueError(f"{name} must be a tensor on {first.device}")
    raise ValueError("the operands must be CUDA (HIP) tensors of one device")


def _elsewhere(index, stream):
    """The context a call has to move into: that of an explicit stream, or of
    a device other than the current one; None where the call already is."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
        return torch.cuda.stream(stream)
    if index != _current_device():
        return torch.cuda.device(index)
    return None


def _raw_stream(index):
    if _raw_stream_of is not None:
        return _raw_stream_of(index)
    return torch.cuda.current_stream(index).cuda_stream


def _mat(t, name, rows=None, cols=None, dtype=None):
    """Checks a 2-D row-major matrix (None: any); returns its row pitch in
    elements (any pitch describes a single row: the shortest that the C
    boundary takes)."""
    size = t.shape
    if len(size) != 2 or (rows is not None and size[0] != rows) or (cols is not None and size[1] != cols):
        want = f"[{'any' if rows is None else rows}, {'any' if cols is None else cols}]"
        raise ValueError(f"{name} must have shape {want}, got {tuple(size)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    pitch, unit = t.stride()
    if unit != 1 and size[1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if size[0] > 1:
        return pitch
    per = 16 // t.element_size()
    return -(-size[1] // per) * per


def _vec(t, name, count, dtype=None):
    """Checks a contiguous vector."""
    size = t.shape
    if len(size) != 1 or size[0] != count or (count > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {count} elements, got shape {tuple(size)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _weight(t, name, count):
    """Pointer and dtype code of an optional weight vector."""
    if t is None:
        return None, 0
    return _vec(t, name, count).data_ptr(), _dt(t, name)


def _scratch(workspace, need, device):
    """Pointer and size of the caller's scratch tensor, or of a new one (kept
    alive by the third value until the launch)."""
    if workspace is None:
        workspace = _empty((need or 16,), (1,), dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def tp_rmsnorm_rotate(x, gamma=None, eps=1e-6, residual=None, rotate=True, out_kind="i8", out=None, scales=None,
                      sum_out=None, stream=None):
    """t = x + residual (fp32, rounded to the residual's dtype) or x; the RMS
    norm of t's rows times gamma, rotated per 256-group (unless rotate=False),
    as int8 codes with one fp32 scale per row (out_kind "i8") or as bf16 rows
    ("bf16"). Returns (codes, scales) or rows; with a residual also t, the new
    stream: (codes, scales, t) or (rows, t). sum_out may be residual (or x)
    itself."""
    index = _device(x, "gamma residual out scales sum_out", (gamma, residual, out, scales, sum_out))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_rmsnorm_rotate(x, gamma, eps, residual, rotate, out_kind, out, scales, sum_out)
    if out_kind not in _KIND:
        raise ValueError("out_kind must be 'i8' or 'bf16'")
    kind, y_dtype = _KIND[out_kind]
    ldx = _mat(x, "x")
    m, k = x.shape
    device = x.device
    g_ptr, g_dt = _weight(gamma, "gamma", k)
    r_ptr = s_ptr = sc_ptr = None
    ldr = lds = s_dt = 0
    if residual is not None:
        ldr = _mat(residual, "residual", m, k)
        s_dt = _dt(residual, "residual")
        if sum_out is None:
            sum_out, lds = _empty((m, k), (k, 1), dtype=residual.dtype, device=device), k
        else:
            lds = _mat(sum_out, "sum_out", m, k, residual.dtype)
        r_ptr, s_ptr = residual.data_ptr(), sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if out is None:
        out, ldy = _empty((m, k), (k, 1), dtype=y_dtype, device=device), k
    else:
        ldy = _mat(out, "out", m, k, y_dtype)
    if kind == TP_NORM_OUT_I8:
        if scales is None:
            scales = _empty((m,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(scales, "scales", m, torch.float32)
        sc_ptr = scales.data_ptr()
    elif scales is not None:
        raise ValueError("scales belong to out_kind 'i8'")
    _lib.check(_lib.load().tp_rmsnorm_rotate(
        x.data_ptr(), _dt(x, "x"), ldx, r_ptr, ldr, s_ptr, lds, s_dt, g_ptr, g_dt, eps,
        TP_A_ROTATE if rotate else TP_A_PREROTATED, m, k, kind, out.data_ptr(), ldy, sc_ptr, _raw_stream(index)))
    if kind == TP_NORM_OUT_I8:
        return (out, scales) if residual is None else (out, scales, sum_out)
    return out if residual is None else (out, sum_out)


def tp_rmsnorm_backward_workspace_size(m, k):
    """Bytes of workspace tp_rmsnorm_rotate_backward needs for dgamma."""
    return _lib.load().tp_rmsnorm_backward_workspace_size(m, k)


def tp_rmsnorm_rotate_backward(dy, t, gamma=None, eps=1e-6, dsum=None, rotate=True, dx_dtype=None, want_dgamma=True,
                               dx=None, dgamma=None, workspace=None, stream=None):
    """Gradients of tp_rmsnorm_rotate (quantization straight through): dy is
    the gradient of its rows (rotated ones unless rotate=False), t its sum (or
    x), dsum the gradient that reaches the stream from behind. Returns
    (dx, dgamma); dgamma is None where it is not wanted. dx (default dtype:
    dsum's, else t's) may be dsum or dy itself."""
    index = _device(dy, "t gamma dsum dx dgamma workspace", (t, gamma, dsum, dx, dgamma, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_rmsnorm_rotate_backward(dy, t, gamma, eps, dsum, rotate, dx_dtype, want_dgamma, dx, dgamma,
                                              workspace)
    lddy = _mat(dy, "dy")
    m, k = dy.shape
    device = dy.device
    ldt = _mat(t, "t", m, k)
    g_ptr, g_dt = _weight(gamma, "gamma", k)
    if dx is None:
        dx = _empty((m, k), (k, 1), dtype=dx_dtype or (t if dsum is None else dsum).dtype, device=device)
        lddx = k
    else:
        lddx = _mat(dx, "dx", m, k, dx_dtype)
    ds_ptr, ldds = None, 0
    if dsum is not None:
        ds_ptr, ldds = dsum.data_ptr(), _mat(dsum, "dsum", m, k, dx.dtype)
    dg_ptr = ws_ptr = ws = None
    ws_bytes = 0
    if want_dgamma or dgamma is not None:
        if dgamma is None:
            dgamma = _empty((k,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(dgamma, "dgamma", k, torch.float32)
        dg_ptr = dgamma.data_ptr()
        ws_ptr, ws_bytes, ws = _scratch(workspace, tp_rmsnorm_backward_workspace_size(m, k), device)
    _lib.check(_lib.load().tp_rmsnorm_rotate_backward(
        dy.data_ptr(), _dt(dy, "dy"), lddy, TP_A_ROTATE if rotate else TP_A_PREROTATED, t.data_ptr(), _dt(t, "t"),
        ldt, g_ptr, g_dt, eps, ds_ptr, ldds, m, k, dx.data_ptr(), _dt(dx, "dx"), lddx, dg_ptr, ws_ptr, ws_bytes,
        _raw_stream(index)))
    return dx, dgamma


_T = 64  # floats of a row of T and dT


def tp_lora_down_prequantized_workspace_size(m, k, r):
    """Bytes of workspace tp_lora_down_prequantized needs."""
    return _lib.load().tp_lora_down_prequantized_workspace_size(m, k, r)


def _t_rows(t, name, m, device):
    """fp32 [m, 64] contiguous, allocated where it is not given."""
    if t is None:
        return _empty((m, _T), (_T, 1), dtype=torch.float32, device=device)
    if _mat(t, name, m, _T, torch.float32) != _T:
        raise ValueError(f"{name} must be contiguous")
    return t


def tp_lora_down_prequantized(qa, sa, lora_a, t=None, workspace=None, stream=None):
    """T = sa (qa . lora_a^T) in fp32 rows of 64 (zeros past r): the first half
    of the side path on activations held as int8 codes and scales; lora_a
    [r, k] in the codes' domain. Returns T [m, 64], as tp_lora_down does."""
    index = _device(qa, "sa lora_a t workspace", (sa, lora_a, t, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_lora_down_prequantized(qa, sa, lora_a, t, workspace)
    ldqa = _mat(qa, "qa", dtype=torch.int8)
    m, k = qa.shape
    device = qa.device
    _vec(sa, "sa", m, torch.float32)
    lda = _mat(lora_a, "lora_a", cols=k)
    r = lora_a.shape[0]
    t = _t_rows(t, "t", m, device)
    ws_ptr, ws_bytes, ws = _scratch(workspace, tp_lora_down_prequantized_workspace_size(m, k, r), device)
    _lib.check(_lib.load().tp_lora_down_prequantized(
        qa.data_ptr(), ldqa, sa.data_ptr(), lora_a.data_ptr(), _dt(lora_a, "lora_a"), lda, m, k, r, t.data_ptr(),
        m * _T * 4, ws_ptr, ws_bytes, _raw_stream(index)))
    return t


def tp_lora_grad_workspace_size(m, n, k, r):
    """Bytes of workspace tp_lora_grad_prequantized needs."""
    return _lib.load().tp_lora_grad_workspace_size(m, n, k, r)


def tp_lora_grad_prequantized(dy, qa, sa, t, lora_b, alpha, rotate=False, da=None, db=None, dt=None, workspace=None,
                              stream=None):
    """Gradients of the side path alpha * T . lora_b^T, T = x . lora_a^T, with
    the activations x = sa qa held in 8 bits: (dA, dB, dT) = (dT^T x, alpha
    dy^T T, alpha dy . lora_b), fp32. dA is in the codes' domain, or with
    rotate=True rotated back (the gradient of an un-rotated lora_a); dT [m, 64]
    gives dx = dT . lora_a."""
    index = _device(dy, "qa sa t lora_b da db dt workspace", (qa, sa, t, lora_b, da, db, dt, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_lora_grad_prequantized(dy, qa, sa, t, lora_b, alpha, rotate, da, db, dt, workspace)
    lddy = _mat(dy, "dy")
    m, n = dy.shape
    device = dy.device
    ldqa = _mat(qa, "qa", m, dtype=torch.int8)
    k = qa.shape[1]
    _vec(sa, "sa", m, torch.float32)
    if t is None:
        raise ValueError("t (the forward's T) is needed")
    _t_rows(t, "t", m, device)
    ldb = _mat(lora_b, "lora_b", n)
    r = lora_b.shape[1]
    dt = _t_rows(dt, "dt", m, device)
    ldda, lddb = k, r
    if da is None:
        da = _empty((r, k), (k, 1), dtype=torch.float32, device=device)
    else:
        ldda = _mat(da, "da", r, k, torch.float32)
    if db is None:
        db = _empty((n, r), (r, 1), dtype=torch.float32, device=device)
    else:
        lddb = _mat(db, "db", n, r, torch.float32)
    ws_ptr, ws_bytes, ws = _scratch(workspace, tp_lora_grad_workspace_size(m, n, k, r), device)
    _lib.check(_lib.load().tp_lora_grad_prequantized(
        dy.data_ptr(), _dt(dy, "dy"), lddy, qa.data_ptr(), ldqa, sa.data_ptr(), t.data_ptr(), lora_b.data_ptr(),
        _dt(lora_b, "lora_b"), ldb, alpha, TP_A_ROTATE if rotate else TP_A_PREROTATED, m, n, k, r, dt.data_ptr(),
        da.data_ptr(), ldda, db.data_ptr(), lddb, ws_ptr, ws_bytes, _raw_stream(index)))
    return da, db, dt


_LAYOUT = {"interleaved": TP_ROPE_INTERLEAVED, "halves": TP_ROPE_HALVES}


def _heads(t, name, m, head_dim, dtype=None):
    """Row pitch, width and head count of a [m, heads * head_dim] matrix."""
    ld = _mat(t, name, m, dtype=dtype)
    width = t.shape[1]
    if head_dim < 1 or width % head_dim != 0:
        raise ValueError(f"{name} must have a multiple of {head_dim} columns, got shape {tuple(t.shape)}")
    return ld, width, width // head_dim


def _axis_bytes(pair_axis, pairs):
    """The axis of each pair, a byte each. Integers one by one: bytes() of an
    array is its memory, and of a number that many zeros."""
    if pair_axis is None:
        return bytes(pairs)
    if type(pair_axis) is not bytes:
        try:
            pair_axis = bytes(list(pair_axis))
        except TypeError as e:
            raise TypeError("pair_axis must be a sequence of integers") from e
        except (ValueError, OverflowError) as e:
            raise ValueError("pair_axis must hold axis numbers") from e
    if len(pair_axis) != pairs:
        raise ValueError(f"pair_axis must have {pairs} entries, got {len(pair_axis)}")
    return pair_axis


def _rope_args(m, head_dim, positions, inv_freq, pair_axis, layout, q_gamma, k_gamma, eps):
    """The arguments that forward and backward share, in the C order."""
    if layout not in _LAYOUT:
        raise ValueError("layout must be 'interleaved' or 'halves'")
    qg, g_dt = _weight(q_gamma, "q_gamma", head_dim)
    kg, k_dt = _weight(k_gamma, "k_gamma", head_dim)
    if qg is None:
        g_dt = k_dt
    elif kg is not None and g_dt != k_dt:
        raise TypeError("q_gamma and k_gamma must have one dtype")
    pairs = 0 if inv_freq is None else inv_freq.shape[0]
    if pairs == 0:
        return qg, kg, g_dt, eps, None, 0, 1, None, None, 0, _LAYOUT[layout]
    if positions is None:
        raise ValueError("positions are needed")
    if positions.dim() == 1:
        positions = positions[:, None]
    ldpos = _mat(positions, "positions", m, dtype=torch.int32)
    _vec(inv_freq, "inv_freq", pairs, torch.float32)
    axis = _axis_bytes(pair_axis, pairs)
    return (qg, kg, g_dt, eps, positions.data_ptr(), ldpos, positions.shape[1], inv_freq.data_ptr(), axis, pairs,
            _LAYOUT[layout])


def tp_qk_norm_rope(q, k, head_dim, positions=None, inv_freq=None, pair_axis=None, layout="interleaved", q_gamma=None,
                    k_gamma=None, eps=1e-6, out_dtype=None, q_out=None, k_out=None, stream=None):
    """The RMS norm of each head of q and k (where its gamma is given), then
    rotary positions. q, k [m, heads * head_dim] (views of one qkv output, of
    different head counts); positions int32 [m, axes] (or [m]); inv_freq fp32
    [pairs]; pair_axis the axis of each pair (host integers, default all 0);
    layout "interleaved" (pairs of neighbours) or "halves". Columns past the
    rotated ones are passed on. Returns (q_out, k_out), which may be the inputs
    themselves; default dtype: the inputs'."""
    index = _device(q, "k positions inv_freq q_gamma k_gamma q_out k_out",
                    (k, positions, inv_freq, q_gamma, k_gamma, q_out, k_out))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_qk_norm_rope(q, k, head_dim, positions, inv_freq, pair_axis, layout, q_gamma, k_gamma, eps,
                                   out_dtype, q_out, k_out)
    m, x_dtype, device = q.shape[0], q.dtype, q.device
    ldq, wq, hq = _heads(q, "q", m, head_dim)
    ldk, wk, hk = _heads(k, "k", m, head_dim, x_dtype)
    shared = _rope_args(m, head_dim, positions, inv_freq, pair_axis, layout, q_gamma, k_gamma, eps)
    if out_dtype is None:
        out_dtype = x_dtype if q_out is None else q_out.dtype
    ldqo, ldko = wq, wk
    if q_out is None:
        q_out = _empty((m, wq), (wq, 1), dtype=out_dtype, device=device)
    else:
        ldqo = _mat(q_out, "q_out", m, wq, out_dtype)
    if k_out is None:
        k_out = _empty((m, wk), (wk, 1), dtype=out_dtype, device=device)
    else:
        ldko = _mat(k_out, "k_out", m, wk, out_dtype)
    _lib.check(_lib.load().tp_qk_norm_rope(
        q.data_ptr(), ldq, k.data_ptr(), ldk, _dt(q, "q"), m, hq, hk, head_dim, *shared, q_out.data_ptr(), ldqo,
        k_out.data_ptr(), ldko, _dt(q_out, "q_out"), _raw_stream(index)))
    return q_out, k_out


def tp_qk_norm_rope_workspace_size(m, heads_q, heads_k, head_dim):
    """Bytes of workspace tp_qk_norm_rope_backward needs for the weights' gradients."""
    return _lib.load().tp_qk_norm_rope_workspace_size(m, heads_q, heads_k, head_dim)


def _normed(x, gamma, like, name):
    """Pointer, pitch and dtype code of a normed tensor's input."""
    if gamma is None:
        return None, 0, None
    if x is None:
        raise ValueError(f"{name} is needed for the gradient of its norm")
    return x.data_ptr(), _mat(x, name, like.shape[0], like.shape[1]), _dt(x, name)


def tp_qk_norm_rope_backward(dq_out, dk_out, q, k, head_dim, positions=None, inv_freq=None, pair_axis=None,
                             layout="interleaved", q_gamma=None, k_gamma=None, eps=1e-6, dx_dtype=None,
                             want_dgamma=True, dq=None, dk=None, dq_gamma=None, dk_gamma=None, workspace=None,
                             stream=None):
    """Gradients of tp_qk_norm_rope: (dq, dk, dq_gamma, dk_gamma), the latter
    None for a tensor without a norm or where want_dgamma is False. q and k (the
    forward's inputs) may be None for a tensor without a norm. Default dtype of
    dq and dk: dq_out's."""
    index = _device(dq_out, "dk_out q k positions inv_freq q_gamma k_gamma dq dk dq_gamma dk_gamma workspace",
                    (dk_out, q, k, positions, inv_freq, q_gamma, k_gamma, dq, dk, dq_gamma, dk_gamma, workspace))
    scope = _elsewhere(index, stream)
    if scope is not None:
        with scope:
            return tp_qk_norm_rope_backward(dq_out, dk_out, q, k, head_dim, positions, inv_freq, pair_axis, layout,
                                            q_gamma, k_gamma, eps, dx_dtype, want_dgamma, dq, dk, dq_gamma, dk_gamma,
                                            workspace)
    m, y_dtype, device = dq_out.shape[0], dq_out.dtype, dq_out.device
    lddqo, wq, hq = _heads(dq_out, "dq_out", m, head_dim)
    lddko, wk, hk = _heads(dk_out, "dk_out", m, head_dim, y_dtype)
    shared = _rope_args(m, head_dim, positions, inv_freq, pair_axis, layout, q_gamma, k_gamma, eps)
    q_ptr, ldq, q_dt = _normed(q, q_gamma, dq_out, "q")
    k_ptr, ldk, k_dt = _normed(k, k_gamma, dk_out, "k")
    if q_dt is None:
        q_dt = k_dt
    elif k_dt is not None and q_dt != k_dt:
        raise TypeError("q and k must have one dtype")
    if dx_dtype is None:
        dx_dtype = y_dtype if dq is None else dq.dtype
    lddq, lddk = wq, wk
    if dq is None:
        dq = _empty((m, wq), (wq, 1), dtype=dx_dtype, device=device)
    else:
        lddq = _mat(dq, "dq", m, wq, dx_dtype)
    if dk is None:
        dk = _empty((m, wk), (wk, 1), dtype=dx_dtype, device=device)
    else:
        lddk = _mat(dk, "dk", m, wk, dx_dtype)
    if (q_gamma is None and dq_gamma is not None) or (k_gamma is None and dk_gamma is not None):
        raise ValueError("the gradient of a weight that is not given")
    dqg_ptr = dkg_ptr = ws_ptr = ws = None
    ws_bytes = 0
    if q_gamma is not None and (want_dgamma or dq_gamma is not None):
        if dq_gamma is None:
            dq_gamma = _empty((head_dim,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(dq_gamma, "dq_gamma", head_dim, torch.float32)
        dqg_ptr = dq_gamma.data_ptr()
    if k_gamma is not None and (want_dgamma or dk_gamma is not None):
        if dk_gamma is None:
            dk_gamma = _empty((head_dim,), (1,), dtype=torch.float32, device=device)
        else:
            _vec(dk_gamma, "dk_gamma", head_dim, torch.float32)
        dkg_ptr = dk_gamma.data_ptr()
    if dq_gamma is not None or dk_gamma is not None:
        ws_ptr, ws_bytes, ws = _scratch(workspace, tp_qk_norm_rope_workspace_size(m, hq, hk, head_dim), device)
    _lib.check(_lib.load().tp_qk_norm_rope_backward(
        dq_out.data_ptr(), lddqo, dk_out.data_ptr(), lddko, _dt(dq_out, "dq_out"), q_ptr, ldq, k_ptr, ldk, q_dt or 0,
        m, hq, hk, head_dim, *shared, dq.data_ptr(), lddq, dk.data_ptr(), lddk, _dt(dq, "dq"), dqg_ptr, dkg_ptr,
        ws_ptr, ws_bytes, _raw_stream(index)))
    return dq, dk, dq_gamma, dk_gamma
