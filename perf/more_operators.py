"""Cases that measure layer norm, dropout and the block-scaled 8-bit float products.

Five operators of a pre-norm block's branches, in serving and in training:

  ln          dropout of the branch, residual addition, layer norm, rotation
              per 256-group, then bf16 rows, int8 codes with a scale per row,
              or 8-bit float codes with a scale per 128 columns of a row
  ln_bwd      its gradients (stream, branch, weight and bias; the incoming
              gradient may be in the rotated domain)
  dropout     x kept or dropped by a counter-based generator, scaled, added to
              a residual; the mask is never stored
  fp8         y = x . w^T with both operands in 8-bit floating point: x is
              quantized in the call (a scale per row and 128 columns), w is
              held as codes with a scale per 128 x 128 block
  fp8_bwd     dx = dy . w and dw = dy^T . x of the same product, dy and x
              quantized in the call along the dimension that is summed

Where `own` is false, run() computes an operator with elementary torch
operations; where it is true, it calls the framework.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
GROUP = 256  # columns that the rotation mixes
BLOCK = 128  # elements that share a scale
E4M3_MAX = 448.0


def listed():
    return [
        # The input of a projection of a 4096-token image in training: the
        # branch's output dropped out, added to the stream, normed, rotated.
        dict(name="ln rows 4096", op="ln", m=4096, k=4096, x="bf16", stream="bf16", residual=True, p=0.1, rotate=True,
             kind="bf16"),
        # The same in front of an 8-bit float product, serving, a wide model's
        # prompt on the fp32 output of the previous projection.
        dict(name="ln fp8 2000", op="ln", m=2000, k=8192, x="f32", stream="bf16", residual=True, p=0.0, rotate=False,
             kind="fp8"),
        # One new token in front of an int8 product: latency.
        dict(name="ln codes 1", op="ln", m=1, k=4096, x="bf16", stream="bf16", residual=True, p=0.0, rotate=True,
             kind="i8"),
        # Training step at 4096 tokens: fp32 gradient out of the projection's
        # backward (still rotated), the branch's dropout undone on the way.
        dict(name="ln_bwd 4096", op="ln_bwd", m=4096, k=4096, dy="f32", t="bf16", dx="bf16", dsum=True, p=0.1,
             rotate=True),
        # A ragged batch in full precision, wide rows, first layer.
        dict(name="ln_bwd 333", op="ln_bwd", m=333, k=12288, dy="f32", t="f32", dx="f32", dsum=False, p=0.0,
             rotate=False),
        # Dropout behind a feed-forward layer's middle, and of a short ragged
        # batch whose rows are no multiple of a vector.
        dict(name="dropout 4096", op="dropout", m=4096, k=12288, x="bf16", y="bf16", residual=True, p=0.1),
        dict(name="dropout 77", op="dropout", m=77, k=1161, x="f32", y="f32", residual=False, p=0.25),
        # A feed-forward layer's first product over 4096 tokens.
        dict(name="fp8 4096", op="fp8", m=4096, n=12288, k=4096, x="bf16", y="bf16", rotate=False),
        # One new token through its second product: latency, the weights' bytes.
        dict(name="fp8 1", op="fp8", m=1, n=4096, k=12288, x="bf16", y="bf16", rotate=False),
        # A few sequences at once, odd output width, rotated, fp32 output.
        dict(name="fp8 33", op="fp8", m=33, n=1163, k=1280, x="f32", y="f32", rotate=True),
        # Both gradients of a square projection over a ragged batch of tokens.
        dict(name="fp8_bwd 2000", op="fp8_bwd", m=2000, n=4096, k=4096, dy="bf16", x="bf16", dx="bf16", rotate=False),
        # A short prompt, full-precision gradients, odd widths.
        dict(name="fp8_bwd 77", op="fp8_bwd", m=77, n=1163, k=1280, dy="f32", x="bf16", dx="f32", rotate=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_bwd", "ln_bwd", "dropout", "fp8", "fp8", "fp8_bwd"])
    dt = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    m = _log_int(rng, 1, 4096)
    if op in ("ln", "ln_bwd"):
        k = GROUP * _log_int(rng, 1, 48)
        c = dict(op=op, m=min(m, 4096 * 4096 // k), k=k)
        p = rng.choice([0.0, 0.05, 0.1, 0.5])
        if op == "ln":
            residual = rng.random() < 0.8
            c.update(x=dt(), stream=dt(), residual=residual, p=p if residual else 0.0, rotate=rng.random() < 0.6,
                     kind=rng.choice(["bf16", "i8", "fp8"]))
        else:
            c.update(dy=dt(), t=dt(), dx=dt(), dsum=rng.random() < 0.7, p=p, rotate=rng.random() < 0.6)
        return c
    if op == "dropout":
        return dict(op=op, m=m, k=_log_int(rng, 1, 12288), x=dt(), y=dt(), residual=rng.random() < 0.5,
                    p=rng.choice([0.01, 0.1, 0.25, 0.5]))
    rotate = rng.random() < 0.4
    n = _log_int(rng, 16, 12288)
    k = 2 * BLOCK * rng.randint(1, 24) if rotate else BLOCK * rng.randint(1, 48)
    if op == "fp8":
        return dict(op=op, m=min(m, max(1, 4096 * 12288 * 4096 // (n * k))), n=n, k=k, x=dt(), y=dt(), rotate=rotate)
    return dict(op=op, m=min(m, max(1, 2000 * 12288 * 4096 // (n * k))), n=n, k=k, dy=dt(), x=dt(), dx=dt(),
                rotate=rotate)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _padded(t):
    """The same matrix with a row pitch that is a multiple of 16 bytes."""
    per = 16 // t.element_size()
    m, k = t.shape
    out = torch.zeros((m, -(-k // per) * per), device="cuda", dtype=t.dtype)
    out[:, :k] = t
    return out[:, :k]


def _rows(g, m, k, dtype):
    """Rows off zero, with a few channels far larger than the rest."""
    x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float32) + 0.25
    big = torch.randint(0, k, (max(1, k // 200),), generator=g, device="cuda")
    x[:, big] *= 30.0
    return _padded(x.to(dtype))


def _sylvester():
    """H / 16, H[i][j] = (-1)^popcount(i & j)."""
    i = torch.arange(GROUP, device="cuda")
    odd = i[:, None] & i[None, :]
    for shift in (4, 2, 1):
        odd = odd ^ (odd >> shift)
    return (1.0 - 2.0 * (odd & 1).double()) / 16.0


def _rng_state(g):
    """Seed and offset of the generator, as a training program keeps them."""
    return torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op, m, k = c["op"], c["m"], c["k"]
    c["h_"] = _sylvester()
    if op in ("ln", "ln_bwd"):
        c["gamma_"] = (1.0 + _randn(g, (k,), torch.float32, 0.1)).to(torch.bfloat16)
        c["beta_"] = _randn(g, (k,), torch.bfloat16, 0.1)
        c["eps"] = 1e-5
    if "p" in c:
        c["rng_"] = _rng_state(g) if c["p"] > 0 else None
    if op == "ln":
        c["x_"] = _rows(g, m, k, _DT[c["x"]])
        c["res_"] = (_randn(g, (m, k), torch.float32, 2.0) + 0.5).to(_DT[c["stream"]]) if c["residual"] else None
    elif op == "ln_bwd":
        c["dy_"] = _randn(g, (m, k), _DT[c["dy"]], 0.02)
        c["t_"] = _rows(g, m, k, _DT[c["t"]])
        c["ds_"] = _randn(g, (m, k), _DT[c["dx"]], 0.02) if c["dsum"] else None
    elif op == "dropout":
        c["x_"] = _rows(g, m, k, _DT[c["x"]])
        c["res_"] = _padded(_randn(g, (m, k), _DT[c["y"]])) if c["residual"] else None
    else:
        n = c["n"]
        w = torch.randn((n, k), generator=g, device="cuda", dtype=torch.float32) * k ** -0.5
        codes, s = _quantize_blocks(w)
        if op == "fp8":
            c["x_"] = _rows(g, m, k, _DT[c["x"]])
            c["w_"], c["ws_"] = codes[:n].to(torch.float8_e4m3fn), s.contiguous()
        else:
            c["x_"] = _rows(g, m, k, _DT[c["x"]])
            c["dy_"] = _padded(_randn(g, (m, n), _DT[c["dy"]], 0.02))
            c["wt_"], c["wts_"] = codes.t().contiguous().to(torch.float8_e4m3fn), s.t().contiguous()
    return c


# --------------------------------------------------------------- plain forms


def _rotate(c, x):
    return (x.reshape(-1, GROUP) @ c["h_"].to(x.dtype)).reshape(x.shape)


def _threshold(p):
    """Of 65536 values of a 16-bit number the lowest so many drop."""
    return int(round(p * 65536))


def _keep(rng, m, k, p):
    """Philox4x32-10 (Salmon and others, 2011): one call for eight elements of
    a row, 16 bits each; key: the seed, counter: the run of eight and the
    offset."""
    runs = -(-k // 8)
    low = 0xFFFFFFFF
    run = torch.arange(m * runs, device="cuda", dtype=torch.int64)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    a, b = run & low, run >> 32
    d, e = (rng[1] & low).expand_as(a), ((rng[1] >> 32) & low).expand_as(a)
    for _ in range(10):
        p0, p1 = a * 0xD2511F53, d * 0xCD9E8D57
        a, b, d, e = ((p1 >> 32) & low) ^ b ^ k0, p1 & low, ((p0 >> 32) & low) ^ e ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, d, e], dim=1)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(m, runs * 8)[:, :k]
    return halves >= _threshold(p)


def _scale(p):
    return float(np.float32(65536.0 / (65536 - _threshold(p))))


def _dropped(x, rng, p):
    """fp32: x / (1 - p) where it is kept, 0 where it is not."""
    x = x.float()
    return torch.where(_keep(rng, x.shape[0], x.shape[1], p), x * _scale(p), torch.zeros_like(x))


def _round_e4m3(q):
    """fp64 values to the nearest of e4m3 (even on a tie), as fp64."""
    e = (torch.frexp(q)[1] - 1).clamp_(min=-6).long()
    step = ((e - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(q / step) * step).clamp_(-E4M3_MAX, E4M3_MAX)


def _codes_by(x, amax):
    """Codes and scales of fp64 values whose blocks have the largest
    magnitudes amax (of x's shape, with ones along the blocks)."""
    s = (amax / E4M3_MAX).float()
    d = torch.where(s > 0, s, torch.ones_like(s)).double()
    return torch.where(s > 0, _round_e4m3(x / d), torch.zeros_like(x)), s


def _pad_to_block(x, dim):
    short = -x.shape[dim] % BLOCK
    if not short:
        return x
    shape = list(x.shape)
    shape[dim] = short
    return torch.cat([x, x.new_zeros(shape)], dim=dim)


def _quantize_rows(x):
    """A scale per row and 128 columns: codes [m, kp], scales [m, kp / 128]."""
    x = _pad_to_block(x.double(), 1)
    y = x.reshape(x.shape[0], -1, BLOCK)
    q, s = _codes_by(y, y.abs().amax(dim=2, keepdim=True))
    return q.reshape(x.shape), s[:, :, 0]


def _quantize_blocks(x):
    """A scale per 128 x 128 block: codes padded to whole blocks."""
    x = _pad_to_block(_pad_to_block(x.double(), 0), 1)
    y = x.reshape(x.shape[0] // BLOCK, BLOCK, x.shape[1] // BLOCK, BLOCK)
    q, s = _codes_by(y, y.abs().amax(dim=(1, 3), keepdim=True))
    return q.reshape(x.shape), s[:, 0, :, 0]


def _by_rows(codes, s):
    """fp32 values of codes with a scale per row and 128 columns."""
    y = codes.float().reshape(codes.shape[0], -1, BLOCK) * s[:, :, None]
    return y.reshape(codes.shape)


def _by_blocks(codes, s):
    """fp32 values of codes with a scale per 128 x 128 block."""
    full = s.repeat_interleave(BLOCK, dim=0).repeat_interleave(BLOCK, dim=1)
    return codes.float() * full[:codes.shape[0], :codes.shape[1]]


def _ln(c):
    t = c["x_"]
    if c["res_"] is not None:
        t = _dropped(t, c["rng_"], c["p"]) if c["p"] > 0 else t.float()
        t = (t + c["res_"].float()).to(_DT[c["stream"]])
    # codes are decided next to rounding borders: 64 bits there
    v = t.float() if c["kind"] == "bf16" else t.double()
    d = v - v.mean(dim=1, keepdim=True)
    h = d * torch.rsqrt(d.square().mean(dim=1, keepdim=True) + c["eps"])
    h = h * c["gamma_"].to(v.dtype) + c["beta_"].to(v.dtype)
    if c["rotate"]:
        h = _rotate(c, h)
    out = {} if c["res_"] is None else {"sum": t}
    if c["kind"] == "bf16":
        out["rows"] = h.to(torch.bfloat16)
    elif c["kind"] == "i8":
        s = (h.abs().amax(dim=1) / 127.0).float()
        out["values"] = torch.round(h / s.double()[:, None]).clamp(-127, 127).float() * s[:, None]
    else:
        out["values"] = _by_rows(*_quantize_rows(h))
    return out


def _ln_bwd(c):
    dy, t, gamma = c["dy_"].float(), c["t_"].float(), c["gamma_"].float()
    g = _rotate(c, dy) if c["rotate"] else dy
    d = t - t.mean(dim=1, keepdim=True)
    r = torch.rsqrt(d.square().mean(dim=1, keepdim=True) + c["eps"])
    n, w = d * r, g * gamma
    dx = r * (w - w.mean(dim=1, keepdim=True) - n * (w * n).mean(dim=1, keepdim=True))
    if c["ds_"] is not None:
        dx = dx + c["ds_"].float()
    out = {"dx": dx.to(_DT[c["dx"]]), "dgamma": (g * n).sum(dim=0), "dbeta": g.sum(dim=0)}
    if c["p"] > 0:
        out["dbranch"] = _dropped(dx, c["rng_"], c["p"]).to(_DT[c["dx"]])
    return out


def _dropout(c):
    y = _dropped(c["x_"], c["rng_"], c["p"])
    if c["res_"] is not None:
        y = y + c["res_"].float()
    return {"y": y.to(_DT[c["y"]])}


def _fp8(c):
    x = c["x_"].double()
    a = _by_rows(*_quantize_rows(_rotate(c, x) if c["rotate"] else x))
    return {"y": (a @ _by_blocks(c["w_"], c["ws_"]).t()).to(_DT[c["y"]])}


def _fp8_bwd(c):
    x, dy, n = c["x_"].double(), c["dy_"], c["n"]
    x = _rotate(c, x) if c["rotate"] else x
    dx = _by_rows(*_quantize_rows(dy)) @ _by_blocks(c["wt_"], c["wts_"]).t()
    dw = _by_rows(*_quantize_rows(dy.t())) @ _by_rows(*_quantize_rows(x.t())).t()
    return {"dx": dx.to(_DT[c["dx"]]), "dw": dw}


_PLAIN = {"ln": _ln, "ln_bwd": _ln_bwd, "dropout": _dropout, "fp8": _fp8, "fp8_bwd": _fp8_bwd}


# -------------------------------------------------------- the framework's calls


def _framework(c):
    import int4_quantized_gemm_amd as tp

    op = c["op"]
    if op == "ln":
        got = tp.tp_layernorm_rotate(c["x_"], c["gamma_"], c["beta_"], eps=c["eps"], residual=c["res_"],
                                     drop_p=c["p"], rng=c["rng_"], rotate=c["rotate"], out_kind=c["kind"])
        if c["kind"] == "bf16":
            out = {"rows": got if c["res_"] is None else got[0]}
        elif c["kind"] == "i8":
            out = {"values": got[0] * got[1][:, None]}  # what the codes stand for
        else:
            y = got[0].float().view(c["m"], -1, BLOCK) * got[1].t()[:, :, None]
            out = {"values": y.view(c["m"], c["k"])}
        if c["res_"] is not None:
            out["sum"] = got[-1]
        return out
    if op == "ln_bwd":
        dx, dbranch, dgamma, dbeta = tp.tp_layernorm_rotate_backward(
            c["dy_"], c["t_"], c["gamma_"], eps=c["eps"], dsum=c["ds_"], drop_p=c["p"], rng=c["rng_"],
            rotate=c["rotate"], dx_dtype=_DT[c["dx"]])
        out = {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        if c["p"] > 0:
            out["dbranch"] = dbranch
        return out
    if op == "dropout":
        return {"y": tp.tp_dropout(c["x_"], c["p"], c["rng_"], residual=c["res_"], out_dtype=_DT[c["y"]])}
    if op == "fp8":
        a, sa = tp.tp_quantize_fp8(c["x_"], rotate=c["rotate"])
        return {"y": tp.tp_qgemm_fp8(a, sa, c["w_"], c["ws_"], out_dtype=_DT[c["y"]])}
    a, sa, at, sat = tp.tp_quantize_fp8(c["dy_"], want="both")
    xt, sxt = tp.tp_quantize_fp8(c["x_"], rotate=c["rotate"], want="cols")
    return {"dx": tp.tp_qgemm_fp8(a, sa, c["wt_"], c["wts_"], out_dtype=_DT[c["dx"]]),
            "dw": tp.tp_qgemm_fp8(at, sat, xt, sxt, b_block_rows=1, out_dtype=torch.float32)}


def run(state):
    return _framework(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work


def work(case):
    c = case
    op, m, k = c["op"], c["m"], c["k"]
    mask = 1 if c.get("p", 0) > 0 else 0
    if op == "ln":
        per = _SIZE[c["x"]] + (2 * _SIZE[c["stream"]] if c["residual"] else 0) + (2 if c["kind"] == "bf16" else 1)
        scales = {"bf16": 0, "i8": 4 * m, "fp8": 4 * m * (k // BLOCK)}[c["kind"]]
        return {"bytes": m * k * per + scales + 4 * k, "flops": m * k * (8 + (8 if c["rotate"] else 0) + 2 * mask)}
    if op == "ln_bwd":
        per = _SIZE[c["dy"]] + _SIZE[c["t"]] + _SIZE[c["dx"]] * (1 + mask + (1 if c["dsum"] else 0))
        return {"bytes": m * k * per + 10 * k, "flops": m * k * (16 + (8 if c["rotate"] else 0) + mask)}
    if op == "dropout":
        per = _SIZE[c["x"]] + _SIZE[c["y"]] * (2 if c["residual"] else 1)
        return {"bytes": m * k * per, "flops": m * k * (2 if c["residual"] else 1)}
    n = c["n"]
    w = n * k + 4 * -(-n // BLOCK) * (k // BLOCK)
    if op == "fp8":
        return {"bytes": m * k * _SIZE[c["x"]] + w + m * n * _SIZE[c["y"]], "flops": 2 * m * n * k}
    return {"bytes": m * n * _SIZE[c["dy"]] + m * k * (_SIZE[c["x"]] + _SIZE[c["dx"]]) + w + 4 * n * k,
            "flops": 4 * m * n * k}


# -------------------------------------------------------------------- exact


def _butterfly(x):
    """x . blockdiag(H / 16), bit by bit of the column index."""
    shape = x.shape
    x = x.reshape(-1, GROUP)
    for bit in range(8):
        h = 1 << bit
        y = x.reshape(-1, GROUP // (2 * h), 2, h)
        lo, hi = y[:, :, 0], y[:, :, 1]
        x = torch.stack([lo + hi, lo - hi], dim=2).reshape(-1, GROUP)
    return (x / 16.0).reshape(shape)


def _mask64(c, m, k):
    """1 / (1 - p) or 0 for every element, from 64-bit integers on the host."""
    seed, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in c["rng_"].cpu())
    runs = (k + 7) // 8
    word, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    i = np.arange(m * runs, dtype=np.uint64)
    ctr = [i & word, i >> shift, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    for r in range(10):
        ka, kb = ((seed + r * 0x9E3779B9) & 0xFFFFFFFF), (((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        x, y = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(y >> shift) ^ ctr[1] ^ np.uint64(ka), y & word, (x >> shift) ^ ctr[3] ^ np.uint64(kb), x & word]
    bits = np.stack(ctr, axis=1).astype(np.uint32).view(np.uint16).reshape(m, runs * 8)[:, :k]
    t = _threshold(c["p"])
    kept = torch.from_numpy((bits >= t).astype(np.uint8)).cuda()
    return kept.double() * float(np.float32(65536.0 / (65536 - t)))


def _e4m3_table():
    """The magnitudes that codes 0 .. 126 stand for, in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], device="cuda", dtype=torch.float64)


def _values64(x, blocks):
    """What e4m3 codes of x stand for; blocks(x) brings the elements that share
    a scale together in the last dimension."""
    y = blocks(x)
    s = (y.abs().max(dim=-1, keepdim=True).values / E4M3_MAX).float().double()
    table = _e4m3_table()
    mid = (table[1:] + table[:-1]) / 2
    q = (y / torch.where(s > 0, s, torch.ones_like(s))).contiguous()
    at = torch.bucketize(q.abs(), mid)  # a tie counts as the lower code
    tie = (at < 126) & (mid[at.clamp(max=125)] == q.abs())
    at = at + (tie & (at % 2 == 1))
    return torch.where(s > 0, table[at] * q.sign() * s, torch.zeros_like(q))


def _rows64(x):
    """Rows by 128 columns, the last ones filled up with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK))
    return _values64(x, lambda v: v.reshape(v.shape[0], -1, BLOCK)).reshape(x.shape)


def _blocks64(codes, s):
    n, k = codes.shape
    i, j = torch.arange(n, device="cuda") // BLOCK, torch.arange(k, device="cuda") // BLOCK
    return codes.to(torch.float32).double() * s.double()[i][:, j]


def exact(case, seed):
    c = prepare(case, seed)
    op, m, k = c["op"], c["m"], c["k"]
    if op == "ln":
        t = c["x_"].double()
        if c["res_"] is not None:  # the stream is an fp32 sum rounded to its type, by definition
            if c["p"] > 0:
                t = (t * _mask64(c, m, k)).float()
            t = torch.add(t.float(), c["res_"].float()).to(c["res_"].dtype).double()
        mean = t.sum(dim=1, keepdim=True) / k
        dev = ((t - mean).pow(2).sum(dim=1, keepdim=True) / k + c["eps"]).sqrt()
        h = (t - mean) / dev * c["gamma_"].double() + c["beta_"].double()
        h = _butterfly(h) if c["rotate"] else h
        out = {} if c["res_"] is None else {"sum": t}
        if c["kind"] == "bf16":
            out["rows"] = h
        elif c["kind"] == "i8":
            s = (h.abs().max(dim=1).values / 127.0).float().double()[:, None]
            out["values"] = (h / s).round().clamp(-127, 127) * s
        else:
            out["values"] = _rows64(h)
        return out
    if op == "ln_bwd":
        dy, t, gamma = c["dy_"].double(), c["t_"].double(), c["gamma_"].double()
        g = _butterfly(dy) if c["rotate"] else dy
        mean = t.sum(dim=1, keepdim=True) / k
        dev = ((t - mean).pow(2).sum(dim=1, keepdim=True) / k + c["eps"]).sqrt()
        n = (t - mean) / dev
        w = g * gamma
        dx = (w - w.sum(dim=1, keepdim=True) / k - n * ((w * n).sum(dim=1, keepdim=True) / k)) / dev
        if c["ds_"] is not None:
            dx = dx + c["ds_"].double()
        out = {"dx": dx, "dgamma": (g * n).sum(dim=0), "dbeta": g.sum(dim=0)}
        if c["p"] > 0:
            out["dbranch"] = dx * _mask64(c, m, k)
        return out
    if op == "dropout":
        y = c["x_"].double() * _mask64(c, m, k)
        return {"y": y if c["res_"] is None else y + c["res_"].double()}
    x = c["x_"].double()
    x = _butterfly(x) if c["rotate"] else x
    if op == "fp8":
        return {"y": _rows64(x) @ _blocks64(c["w_"], c["ws_"]).t().contiguous()}
    dy = c["dy_"].double()
    dw = _rows64(dy.t().contiguous()) @ _rows64(x.t().contiguous()).t().contiguous()
    return {"dx": _rows64(dy) @ _blocks64(c["wt_"], c["wts_"]).t().contiguous(), "dw": dw}
