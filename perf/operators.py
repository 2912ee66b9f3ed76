"""Cases that measure the operators around the quantized projections of a transformer block.

Six operators, in serving and in the training of LoRA adapters on the frozen
8-bit base:

  norm        residual addition, RMS norm, rotation per 256-group, then int8
              codes with one scale per row, or bf16 rows
  norm_bwd    its gradients (input and weight; the incoming gradient may be in
              the rotated domain, as the projection's backward leaves it)
  side        T = x . lora_a^T from an activation kept as int8 codes and scales
  side_bwd    the gradients of lora_a and lora_b (and of T) from those codes
  rope        per-head RMS norm of q and k, then rotary positions with one to
              four axes (time, height, width)
  rope_bwd    its gradients

Where `own` is false, run() computes an operator with elementary torch
operations; where it is true, it calls the framework.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
GROUP = 256
T_PITCH = 64  # rows of the side path's T are 64 floats, zeros past the rank


def listed():
    return [
        # The input of a bf16-operand projection of a 4096-token image: the
        # residual stream plus the attention's output, normed and rotated.
        dict(name="norm rows 4096", op="norm", m=4096, k=3072, x="bf16", stream="bf16", residual=True, rotate=True,
             kind="bf16"),
        # The same in front of the int8 x int8 product of a 1344x768 image, on
        # the fp32 output of the previous projection.
        dict(name="norm codes 4032", op="norm", m=4032, k=3072, x="f32", stream="bf16", residual=True, rotate=True,
             kind="i8"),
        # One new token: latency.
        dict(name="norm codes 1", op="norm", m=1, k=4096, x="bf16", stream="bf16", residual=True, rotate=True,
             kind="i8"),
        # Training step at 4096 tokens: fp32 gradient out of the projection's
        # backward (still rotated), bf16 stream and stream gradient.
        dict(name="norm_bwd 4096", op="norm_bwd", m=4096, k=3072, dy="f32", t="bf16", dx="bf16", dsum=True,
             rotate=True),
        # A ragged prompt batch in full precision, wide rows, first layer (no
        # gradient arrives at the stream).
        dict(name="norm_bwd 333", op="norm_bwd", m=333, k=12288, dy="f32", t="f32", dx="f32", dsum=False,
             rotate=False),
        # The adapter's first half on the codes the int8 product reads.
        dict(name="side 4096", op="side", m=4096, k=12288, r=32, a="bf16"),
        # Adapter gradients of the qkv projection at 4096 tokens.
        dict(name="side_bwd 4096", op="side_bwd", m=4096, n=9216, k=3072, r=32, dy="bf16", b="bf16", rotate=True),
        # A short prompt, full-precision gradients, output width not a
        # multiple of any tile.
        dict(name="side_bwd 77", op="side_bwd", m=77, n=1160, k=1280, r=8, dy="f32", b="f32", rotate=False),
        # q and k of a 4096-token image out of the fp32 qkv projection, three
        # axes, interleaved pairs, normed heads.
        dict(name="rope 4096", op="rope", m=4096, hq=24, hk=24, d=128, axes=3, pairs=64, layout="interleaved",
             x="f32", out="bf16", norm=True, far=0),
        # One new token deep in a long context, shared key heads, one axis,
        # halves layout, a partial rotation.
        dict(name="rope 1", op="rope", m=1, hq=32, hk=8, d=128, axes=1, pairs=32, layout="halves", x="bf16",
             out="bf16", norm=False, far=1000000),
        dict(name="rope_bwd 4096", op="rope_bwd", m=4096, hq=24, hk=24, d=128, axes=3, pairs=64,
             layout="interleaved", x="bf16", dy="bf16", dx="bf16", norm=True, far=0),
        # A ragged batch, odd head count, narrow heads, full precision.
        dict(name="rope_bwd 515", op="rope_bwd", m=515, hq=7, hk=1, d=80, axes=2, pairs=16, layout="halves",
             x="f32", dy="f32", dx="f32", norm=True, far=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "side", "side_bwd", "side_bwd", "rope", "rope_bwd"])
    dt = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    m = _log_int(rng, 1, 4096)
    if op == "norm":
        k = GROUP * _log_int(rng, 1, 48)
        return dict(op=op, m=min(m, 4096 * 3072 // k), k=k, x=dt(), stream=dt(), residual=rng.random() < 0.7,
                    rotate=rng.random() < 0.8, kind=rng.choice(["i8", "bf16"]))
    if op == "norm_bwd":
        k = GROUP * _log_int(rng, 1, 48)
        return dict(op=op, m=min(m, 4096 * 3072 // k), k=k, dy=dt(), t=dt(), dx=dt(), dsum=rng.random() < 0.7,
                    rotate=rng.random() < 0.7)
    if op == "side":
        return dict(op=op, m=m, k=GROUP * rng.randint(1, 48), r=rng.choice([1, 4, 8, 13, 16, 24, 32, 64]), a=dt())
    if op == "side_bwd":
        r = rng.choice([1, 4, 8, 13, 16, 24, 32, 64])
        return dict(op=op, m=min(m, 4096 * 32 // max(r, 32)), n=8 * _log_int(rng, 4, 1152),
                    k=GROUP * rng.randint(1, 12), r=r, dy=dt(), b=dt(), rotate=rng.random() < 0.5)
    d = rng.choice([64, 80, 96, 128, 128, 256])
    pairs = 4 * rng.randint(1, d // 8)
    c = dict(op=op, m=_log_int(rng, 1, 2048), hq=rng.randint(1, 24), hk=rng.randint(1, 8), d=d,
             axes=rng.randint(1, 4), pairs=pairs, layout=rng.choice(["interleaved", "halves"]), x=dt(),
             norm=rng.random() < 0.6, far=rng.choice([0, 4096, 131072, 1000000]))
    if op == "rope":
        c["out"] = dt()
    else:
        c.update(dy=dt(), dx=dt())
    return c


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _rows(g, m, k, dtype):
    """Rows with a few channels far larger than the rest."""
    x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float32)
    big = torch.randint(0, k, (max(1, k // 200),), generator=g, device="cuda")
    x[:, big] *= 30.0
    return x.to(dtype)


def _codes(g, m, k):
    x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float32)
    s = x.abs().amax(dim=1) / 127.0
    return torch.round(x / s[:, None]).clamp_(-127, 127).to(torch.int8), s


def _pair_axis(pairs, axes):
    """A quarter of the pairs for the first axis, the rest shared evenly."""
    if axes == 1:
        return [0] * pairs
    first = max(1, pairs // 4)
    return [0] * first + [1 + (p * (axes - 1)) // (pairs - first) for p in range(pairs - first)]


def _positions(g, m, axes, far):
    """Token i of an image: time 0, row and column centred on zero, or, far
    along, positions that end at `far`."""
    i = torch.arange(m, device="cuda", dtype=torch.int32)
    if far:
        cols = [far - m + i for _ in range(axes)]
    else:
        side = max(1, int(math.isqrt(m)))
        every = [torch.zeros_like(i), i // side - side // 2, i % side - side // 2, i % 7]
        cols = every[:axes] if axes > 1 else [i]
    jitter = torch.randint(0, 3, (axes,), generator=g, device="cuda", dtype=torch.int32)
    return (torch.stack(cols, dim=1) + jitter).contiguous()


def _sylvester():
    """H / 16, H[i][j] = (-1)^popcount(i & j)."""
    i = torch.arange(GROUP, device="cuda")
    odd = i[:, None] & i[None, :]
    for shift in (4, 2, 1):
        odd = odd ^ (odd >> shift)
    return (1.0 - 2.0 * (odd & 1).double()) / 16.0


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op, m = c["op"], c["m"]
    c["h_"] = _sylvester()
    if op == "norm":
        c["x_"] = _rows(g, m, c["k"], _DT[c["x"]])
        c["res_"] = _randn(g, (m, c["k"]), _DT[c["stream"]], 2.0) if c["residual"] else None
        c["gamma_"] = (1.0 + _randn(g, (c["k"],), torch.float32, 0.1)).to(torch.bfloat16)
        c["eps"] = 1e-6
    elif op == "norm_bwd":
        c["dy_"] = _randn(g, (m, c["k"]), _DT[c["dy"]], 0.02)
        c["t_"] = _rows(g, m, c["k"], _DT[c["t"]])
        c["ds_"] = _randn(g, (m, c["k"]), _DT[c["dx"]], 0.02) if c["dsum"] else None
        c["gamma_"] = (1.0 + _randn(g, (c["k"],), torch.float32, 0.1)).to(torch.bfloat16)
        c["eps"] = 1e-6
    elif op == "side":
        c["qa_"], c["sa_"] = _codes(g, m, c["k"])
        c["a_"] = _padded(g, (c["r"], c["k"]), _DT[c["a"]], c["k"] ** -0.5)
    elif op == "side_bwd":
        c["qa_"], c["sa_"] = _codes(g, m, c["k"])
        c["dy_"] = _randn(g, (m, c["n"]), _DT[c["dy"]], 0.02)
        c["b_"] = _padded(g, (c["n"], c["r"]), _DT[c["b"]], 0.05)
        t = torch.zeros((m, T_PITCH), device="cuda")
        t[:, :c["r"]] = _randn(g, (m, c["r"]), torch.float32)
        c["tt_"] = t
        c["alpha"] = 2.0
    else:
        d, pairs = c["d"], c["pairs"]
        xt = _DT[c["x"]]
        width = (c["hq"] + c["hk"]) * d
        qk = _randn(g, (m, width), xt, 1.5)
        c["q_"], c["k_"] = qk[:, :c["hq"] * d], qk[:, c["hq"] * d:]
        c["pos_"] = _positions(g, m, c["axes"], c["far"])
        c["freq_"] = (10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float()
        c["axis_"] = _pair_axis(pairs, c["axes"])
        c["axis_dev_"] = torch.tensor(c["axis_"], device="cuda", dtype=torch.int64)
        c["qg_"] = (1.0 + _randn(g, (d,), torch.float32, 0.1)).to(torch.bfloat16) if c["norm"] else None
        c["kg_"] = (1.0 + _randn(g, (d,), torch.float32, 0.1)).to(torch.bfloat16) if c["norm"] else None
        c["eps"] = 1e-6
        if op == "rope_bwd":
            dqk = _randn(g, (m, width), _DT[c["dy"]], 0.02)
            c["dq_"], c["dk_"] = dqk[:, :c["hq"] * d], dqk[:, c["hq"] * d:]
    return c


def _padded(g, shape, dtype, scale):
    """A matrix whose row pitch is a multiple of 16 bytes."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    pitch = -(-shape[1] // per) * per
    return _randn(g, (shape[0], pitch), dtype, scale)[:, :shape[1]]


# --------------------------------------------------------------- plain forms


def _rotate(c, x):
    return (x.reshape(-1, GROUP) @ c["h_"].to(x.dtype)).reshape(x.shape)


def _stream_sum(c):
    if c["res_"] is None:
        return c["x_"]
    return (c["x_"].float() + c["res_"].float()).to(_DT[c["stream"]])


def _norm(c):
    t = _stream_sum(c)
    # 64 bits: the codes are decided next to rounding borders
    t64 = t.double()
    h = t64 * torch.rsqrt(t64.square().mean(dim=1, keepdim=True) + c["eps"]) * c["gamma_"].double()
    if c["rotate"]:
        h = _rotate(c, h)
    out = {} if c["res_"] is None else {"sum": t}
    if c["kind"] == "bf16":
        out["rows"] = h.to(torch.bfloat16)
        return out
    s = (h.abs().amax(dim=1) / 127.0).float()
    q = torch.round(h / s.double()[:, None]).clamp(-127, 127)
    out["values"] = q.float() * s[:, None]
    return out


def _norm_bwd(c):
    dy, t, gamma = c["dy_"].float(), c["t_"].float(), c["gamma_"].float()
    g = _rotate(c, dy) if c["rotate"] else dy
    rr = torch.rsqrt(t.square().mean(dim=1, keepdim=True) + c["eps"])
    gg = g * gamma
    dx = rr * gg - t * (rr * rr * rr * (gg * t).mean(dim=1, keepdim=True))
    if c["ds_"] is not None:
        dx = dx + c["ds_"].float()
    return {"dx": dx.to(_DT[c["dx"]]), "dgamma": (g * t * rr).sum(dim=0)}


def _side(c):
    t = torch.zeros((c["m"], T_PITCH), device="cuda")
    t[:, :c["r"]] = (c["qa_"].float() @ c["a_"].float().t()) * c["sa_"][:, None]
    return {"t": t}


def _side_bwd(c):
    dy, b = c["dy_"].float(), c["b_"].float()
    r = c["r"]
    dt = torch.zeros((c["m"], T_PITCH), device="cuda")
    dt[:, :r] = c["alpha"] * (dy @ b)
    da = (dt[:, :r] * c["sa_"][:, None]).t() @ c["qa_"].float()
    if c["rotate"]:
        da = _rotate(c, da)
    return {"da": da, "db": c["alpha"] * (dy.t() @ c["tt_"][:, :r]), "dt": dt}


def _cos_sin(c):
    angle = c["pos_"].double()[:, c["axis_dev_"]] * c["freq_"].double()
    return angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]


def _pairs_of(c, x):
    """The two members of each rotated pair, and the rest of the head."""
    p = c["pairs"]
    if c["layout"] == "halves":
        return x[..., :p], x[..., p:2 * p], x[..., 2 * p:]
    y = x[..., :2 * p].reshape(x.shape[:-1] + (p, 2))
    return y[..., 0], y[..., 1], x[..., 2 * p:]


def _join(c, a, b, rest):
    if c["layout"] == "halves":
        return torch.cat([a, b, rest], dim=-1)
    return torch.cat([torch.stack([a, b], dim=-1).flatten(-2), rest], dim=-1)


def _rope_heads(c, x, gamma, cos, sin):
    m, width = x.shape
    x = x.float().reshape(m, -1, c["d"])
    if gamma is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + c["eps"]) * gamma.float()
    a, b, rest = _pairs_of(c, x)
    return _join(c, a * cos - b * sin, a * sin + b * cos, rest).reshape(m, width).to(_DT[c["out"]])


def _rope(c):
    cos, sin = _cos_sin(c)
    return {"q": _rope_heads(c, c["q_"], c["qg_"], cos, sin), "k": _rope_heads(c, c["k_"], c["kg_"], cos, sin)}


def _rope_bwd_heads(c, dy, x, gamma, cos, sin):
    m, width = dy.shape
    a, b, rest = _pairs_of(c, dy.float().reshape(m, -1, c["d"]))
    g = _join(c, a * cos + b * sin, b * cos - a * sin, rest)
    dgamma = None
    if gamma is not None:
        x = x.float().reshape(m, -1, c["d"])
        rr = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + c["eps"])
        dgamma = (g * x * rr).sum(dim=(0, 1))
        gg = g * gamma.float()
        g = rr * gg - x * (rr * rr * rr * (gg * x).mean(dim=-1, keepdim=True))
    return g.reshape(m, width).to(_DT[c["dx"]]), dgamma


def _rope_bwd(c):
    cos, sin = _cos_sin(c)
    dq, dqg = _rope_bwd_heads(c, c["dq_"], c["q_"], c["qg_"], cos, sin)
    dk, dkg = _rope_bwd_heads(c, c["dk_"], c["k_"], c["kg_"], cos, sin)
    return {"dq": dq, "dk": dk, **({"dq_gamma": dqg, "dk_gamma": dkg} if c["norm"] else {})}


_PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "side": _side, "side_bwd": _side_bwd, "rope": _rope,
          "rope_bwd": _rope_bwd}


# -------------------------------------------------------- the framework's calls


def _framework(c):
    import int4_quantized_gemm_amd as tp

    op = c["op"]
    if op == "norm":
        got = tp.tp_rmsnorm_rotate(c["x_"], c["gamma_"], eps=c["eps"], residual=c["res_"], rotate=c["rotate"],
                                   out_kind=c["kind"])
        if c["kind"] == "i8":
            out = {"values": got[0] * got[1][:, None]}  # what the codes stand for
        else:
            out = {"rows": got if c["res_"] is None else got[0]}
        if c["res_"] is not None:
            out["sum"] = got[-1]
        return out
    if op == "norm_bwd":
        dx, dgamma = tp.tp_rmsnorm_rotate_backward(c["dy_"], c["t_"], c["gamma_"], eps=c["eps"], dsum=c["ds_"],
                                                   rotate=c["rotate"], dx_dtype=_DT[c["dx"]])
        return {"dx": dx, "dgamma": dgamma}
    if op == "side":
        return {"t": tp.tp_lora_down_prequantized(c["qa_"], c["sa_"], c["a_"])}
    if op == "side_bwd":
        da, db, dt = tp.tp_lora_grad_prequantized(c["dy_"], c["qa_"], c["sa_"], c["tt_"], c["b_"], c["alpha"],
                                                  rotate=c["rotate"])
        return {"da": da, "db": db, "dt": dt}
    how = dict(head_dim=c["d"], positions=c["pos_"], inv_freq=c["freq_"], pair_axis=c["axis_"], layout=c["layout"],
               q_gamma=c["qg_"], k_gamma=c["kg_"], eps=c["eps"])
    if op == "rope":
        q, k = tp.tp_qk_norm_rope(c["q_"], c["k_"], out_dtype=_DT[c["out"]], **how)
        return {"q": q, "k": k}
    dq, dk, dqg, dkg = tp.tp_qk_norm_rope_backward(c["dq_"], c["dk_"], c["q_"], c["k_"], dx_dtype=_DT[c["dx"]],
                                                   **how)
    out = {"dq": dq, "dk": dk}
    if c["norm"]:
        out.update(dq_gamma=dqg, dk_gamma=dkg)
    return out


def run(state):
    return _framework(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work


def work(case):
    c = case
    op, m = c["op"], c["m"]
    if op == "norm":
        k = c["k"]
        per = _SIZE[c["x"]] + (2 * _SIZE[c["stream"]] if c["residual"] else 0) + (1 if c["kind"] == "i8" else 2)
        scales = 4 * m if c["kind"] == "i8" else 0
        return {"bytes": m * k * per + scales + 2 * k, "flops": m * k * (6 + (8 if c["rotate"] else 0))}
    if op == "norm_bwd":
        k = c["k"]
        per = _SIZE[c["dy"]] + _SIZE[c["t"]] + _SIZE[c["dx"]] * (2 if c["dsum"] else 1)
        return {"bytes": m * k * per + 6 * k, "flops": m * k * (12 + (8 if c["rotate"] else 0))}
    if op == "side":
        k, r = c["k"], c["r"]
        return {"bytes": m * k + 4 * m + r * k * _SIZE[c["a"]] + 4 * T_PITCH * m, "flops": 2 * m * k * r}
    if op == "side_bwd":
        n, k, r = c["n"], c["k"], c["r"]
        read = m * n * _SIZE[c["dy"]] + m * k + 4 * m + 4 * m * r + n * r * _SIZE[c["b"]]
        return {"bytes": read + 4 * (r * k + n * r + T_PITCH * m), "flops": 4 * m * n * r + 2 * m * k * r}
    d, heads = c["d"], c["hq"] + c["hk"]
    small = 4 * m * c["axes"] + 4 * c["pairs"] + (4 * d if c["norm"] else 0)
    if op == "rope":
        per = _SIZE[c["x"]] + _SIZE[c["out"]]
        return {"bytes": m * heads * d * per + small, "flops": m * heads * d * (7 if c["norm"] else 3)}
    per = _SIZE[c["dy"]] + _SIZE[c["dx"]] + (_SIZE[c["x"]] if c["norm"] else 0)
    return {"bytes": m * heads * d * per + small + (8 * d if c["norm"] else 0),
            "flops": m * heads * d * (14 if c["norm"] else 3)}


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


def _turn(c, x, back):
    """Heads x [m, heads, d] in fp64 as complex pairs, times e^(i theta) (or
    its conjugate); theta_p = position on the pair's axis times its frequency."""
    p = c["pairs"]
    pos = torch.stack([c["pos_"][:, a] for a in c["axis_"]], dim=1).double()
    theta = pos * c["freq_"].double()
    w = torch.polar(torch.ones_like(theta), -theta if back else theta)[:, None, :]
    y = x.clone()
    if c["layout"] == "halves":
        z = torch.complex(x[..., :p].contiguous(), x[..., p:2 * p].contiguous()) * w
        y[..., :p], y[..., p:2 * p] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:2 * p:2].contiguous(), x[..., 1:2 * p:2].contiguous()) * w
        y[..., 0:2 * p:2], y[..., 1:2 * p:2] = z.real, z.imag
    return y


def exact(case, seed):
    c = prepare(case, seed)
    op, m = c["op"], c["m"]
    if op == "norm":
        t = c["x_"].double()
        if c["res_"] is not None:  # the stream is an fp32 sum rounded to its type, by definition
            t = torch.add(c["x_"].float(), c["res_"].float()).to(c["res_"].dtype).double()
        rms = ((t * t).sum(dim=1) / c["k"] + c["eps"]).sqrt()
        h = t / rms[:, None] * c["gamma_"].double()
        h = _butterfly(h) if c["rotate"] else h
        out = {} if c["res_"] is None else {"sum": t}
        if c["kind"] == "bf16":
            out["rows"] = h
        else:
            s = (h.abs().max(dim=1).values / 127.0).float().double()[:, None]
            out["values"] = (h / s).round().clamp(-127, 127) * s
        return out
    if op == "norm_bwd":
        dy, t, gamma = c["dy_"].double(), c["t_"].double(), c["gamma_"].double()
        g = _butterfly(dy) if c["rotate"] else dy
        rms = ((t * t).sum(dim=1, keepdim=True) / c["k"] + c["eps"]).sqrt()
        n = t / rms
        w = g * gamma
        dx = (w - n * ((w * n).sum(dim=1, keepdim=True) / c["k"])) / rms
        if c["ds_"] is not None:
            dx = dx + c["ds_"].double()
        return {"dx": dx, "dgamma": (g * n).sum(dim=0)}
    if op == "side":
        x = c["qa_"].double() * c["sa_"].double()[:, None]
        t = x @ c["a_"].double().t().contiguous()
        return {"t": torch.cat([t, t.new_zeros((m, T_PITCH - c["r"]))], dim=1)}
    if op == "side_bwd":
        x = c["qa_"].double() * c["sa_"].double()[:, None]
        dy, r = c["dy_"].double(), c["r"]
        dt = dy @ c["b_"].double().contiguous() * c["alpha"]
        da = dt.t().contiguous() @ x
        db = dy.t().contiguous() @ c["tt_"].double()[:, :r].contiguous() * c["alpha"]
        return {"da": _butterfly(da) if c["rotate"] else da, "db": db,
                "dt": torch.cat([dt, dt.new_zeros((m, T_PITCH - r))], dim=1)}
    out = {}
    for name, heads in (("q", c["hq"]), ("k", c["hk"])):
        x = c[name + "_"].double().reshape(m, heads, c["d"])
        gamma = None if c[name + "g_"] is None else c[name + "g_"].double()
        rms = ((x * x).sum(dim=-1, keepdim=True) / c["d"] + c["eps"]).sqrt()
        if op == "rope":
            y = _turn(c, x if gamma is None else x / rms * gamma, False)
            out[name] = y.reshape(m, heads * c["d"])
            continue
        g = _turn(c, c["d%s_" % name].double().reshape(m, heads, c["d"]), True)
        if gamma is not None:
            n = x / rms
            out["d%s_gamma" % name] = (g * n).sum(dim=(0, 1))
            w = g * gamma
            g = (w - n * ((w * n).sum(dim=-1, keepdim=True) / c["d"])) / rms
        out["d" + name] = g.reshape(m, heads * c["d"])
    return out
