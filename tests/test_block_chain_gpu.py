"""The operators around the projections used together, as a block uses them:
a forward pass through residual + norm + quantization, the int8 product with an
adapter in its store, and the norm and positions of q and k; the way back to the
adapter's, the norm weights' and the stream's gradients. Then the same calls on
other streams and in a captured graph, and on buffers past 2^31 elements."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64, host, rel_fro

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS, ALPHA = 1e-6, 1.5


class Block:
    """Inputs of one attention input: stream, frozen int8 qkv projection, a
    rank-r adapter in the codes' domain, norm weights, positions."""

    def __init__(self, m, k, hq, hk, hd, r, seed, d):
        rng = np.random.default_rng(seed)
        draw = lambda shape, s=1.0: torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(s))  # noqa: E731
        self.m, self.k, self.hq, self.hk, self.hd, self.r = m, k, hq, hk, hd, r
        self.n = (hq + 2 * hk) * hd
        self.x, self.res = draw((m, k)).to(d), draw((m, k), 2.0).to(BF16).to(d)
        self.gamma = (1.0 + draw((k,), 0.1)).to(BF16).to(d)
        self.q, self.s = tp.tp_rotate_quantize_weights(draw((self.n, k), 0.02).to(d), bits=8)
        self.a = draw((r, k), k ** -0.5).to(BF16).to(d)
        pad = -(-r // 8) * 8
        self.b = draw((self.n, pad), 0.05).to(BF16).to(d)[:, :r]
        self.qg, self.kg = ((1.0 + draw((hd,), 0.1)).to(d) for _ in range(2))
        pos = np.stack([np.zeros(m), np.arange(m) // 8, np.arange(m) % 8], axis=1).astype(np.int32)
        self.pos = torch.from_numpy(pos).to(d)
        self.freq = torch.from_numpy((10000.0 ** (-np.arange(hd // 2) / (hd // 2))).astype(np.float32)).to(d)
        self.axis = [0] * (hd // 8) + [1] * (hd // 8) + [2] * (hd // 4)
        self.grad = draw((m, self.n), 0.02).to(d)
        self.dsum = draw((m, k), 0.02).to(BF16).to(d)
        self.cq, self.ck = hq * hd, (hq + hk) * hd
        # the frozen weight's codes by column, for the input's gradient (the
        # product sums over whole 256-groups: zeros fill the last one)
        self.pad = -self.n % 256
        self.qt = torch.nn.functional.pad(self.q.t(), (0, self.pad)).contiguous()
        self.ones = torch.ones((k,), device=d)

    def rope(self):
        return dict(head_dim=self.hd, positions=self.pos, inv_freq=self.freq, pair_axis=self.axis, q_gamma=self.qg,
                    k_gamma=self.kg, eps=EPS)

    def forward(self):
        qa, sa, t = tp.tp_rmsnorm_rotate(self.x, self.gamma, eps=EPS, residual=self.res)
        low = tp.tp_lora_down_prequantized(qa, sa, self.a)
        qkv = tp.tp_qgemm_w8a8_prequantized_lora(qa, sa, self.q, self.s, low, self.b, ALPHA)
        out = qkv.clone()
        tp.tp_qk_norm_rope(out[:, :self.cq], out[:, self.cq:self.ck], q_out=out[:, :self.cq],
                           k_out=out[:, self.cq:self.ck], **self.rope())
        return qa, sa, t, low, qkv, out

    def backward(self, qa, sa, t, low, qkv):
        dy = self.grad.clone()
        _, _, dqg, dkg = tp.tp_qk_norm_rope_backward(
            dy[:, :self.cq], dy[:, self.cq:self.ck], qkv[:, :self.cq], qkv[:, self.cq:self.ck], dq=dy[:, :self.cq],
            dk=dy[:, self.cq:self.ck], **self.rope())
        da, db, dt = tp.tp_lora_grad_prequantized(dy, qa, sa, low, self.b, ALPHA)
        # the input's gradient, in the rotated domain: through the frozen codes
        # (bf16 operand), and through the adapter
        dys = torch.nn.functional.pad(dy * self.s, (0, self.pad)).to(BF16)
        dh = tp.tp_qgemm_w8(dys, self.qt, self.ones, rotate=False, out_dtype=F32)
        dh += dt[:, :self.r] @ self.a.float()
        dx, dgamma = tp.tp_rmsnorm_rotate_backward(dh, t, self.gamma, eps=EPS, dsum=self.dsum)
        return da, db, dqg, dkg, dx, dgamma, dy

    # ------------------------------------------------------ the same in fp64
    def _rope64(self, y):
        pos, freq = self.pos.cpu().numpy(), self.freq.cpu().numpy()
        part = lambda lo, hi, g: oracle.norm_rope(y[:, lo:hi], self.hd, pos, freq, self.axis, False, f64(g), EPS)  # noqa: E731
        return np.concatenate([part(0, self.cq, self.qg), part(self.cq, self.ck, self.kg), y[:, self.ck:]], axis=1)

    def qkv64(self, qa, sa, a, b):
        x = qa.astype(np.float64) * sa.astype(np.float64)[:, None]
        w = host(self.q).astype(np.float64) * f64(self.s)[:, None]
        return x @ w.T + ALPHA * (x @ a.T) @ b.T

    def loss64(self, qa, sa, a, b):
        return float(np.sum(f64(self.grad) * self._rope64(self.qkv64(qa, sa, a, b))))

    def backward64(self, qa, sa, t):
        pos, freq = self.pos.cpu().numpy(), self.freq.cpu().numpy()
        y = self.qkv64(qa, sa, f64(self.a), f64(self.b))
        g = f64(self.grad)
        parts = []
        for lo, hi, gam in ((0, self.cq, self.qg), (self.cq, self.ck, self.kg)):
            parts.append(oracle.norm_rope_backward(g[:, lo:hi], y[:, lo:hi], self.hd, pos, freq, self.axis, False,
                                                   f64(gam), EPS))
        dy = np.concatenate([parts[0][0], parts[1][0], g[:, self.ck:]], axis=1)
        low = oracle.lora_down_codes(qa, sa, f64(self.a))
        da, db, dt = oracle.lora_grad_codes(dy, qa, sa, low, f64(self.b), ALPHA)
        dh = dy @ (host(self.q).astype(np.float64) * f64(self.s)[:, None]) + dt @ f64(self.a)
        dx, dgamma = oracle.rmsnorm_backward(dh, t, f64(self.gamma), EPS, dsum=f64(self.dsum))
        return da, db, parts[0][1], parts[1][1], dx, dgamma


@pytest.mark.parametrize("m,k,hq,hk,hd,r", [(64, 1024, 6, 2, 64, 16), (37, 768, 3, 1, 128, 13)])
def test_block_forward_and_gradients(m, k, hq, hk, hd, r):
    d = dev()
    announce("block forward and backward", m, k, hq, hk, hd, r)
    blk = Block(m, k, hq, hk, hd, r, seed=m, d=d)
    qa, sa, t, low, qkv, out = blk.forward()
    t64 = oracle.stream_sum(f64(blk.x), f64(blk.res), True)
    rq, rs = oracle.quantize_activations_int8(oracle.rmsnorm(t64, f64(blk.gamma), EPS))
    assert np.array_equal(host(qa), rq) and np.array_equal(host(sa), rs) and np.array_equal(f64(t), t64)
    a64, b64 = f64(blk.a), f64(blk.b)
    # fp32 all the way behind the codes: about 100 roundings of 2^-24 on the
    # longest path, each against values of the result's size
    assert rel_fro(f64(out), blk._rope64(blk.qkv64(rq, rs, a64, b64))) <= 1e-5
    got = blk.backward(qa, sa, t, low, qkv)
    want = blk.backward64(rq, rs, t64)
    for name, g, w in zip(("dA", "dB", "dq_gamma", "dk_gamma"), got, want):
        assert rel_fro(f64(g), w) <= 1e-5, name
    # through the frozen weight the gradient is a bf16 operand: 2^-8 a value at
    # most, and dx itself is bf16: another 2^-8
    for name, g, w in zip(("dx", "dgamma"), got[4:], want[4:]):
        assert rel_fro(f64(g), w) <= 2 * B.HALF_BF16, name
    # the adapter's gradients against differences of the loss
    rng = np.random.default_rng(1)
    for i, p in ((0, a64), (1, b64)):
        e = rng.standard_normal(p.shape)
        step = 1e-5 / np.linalg.norm(e)

        def move(h):
            return blk.loss64(rq, rs, a64 + h * e, b64) if i == 0 else blk.loss64(rq, rs, a64, b64 + h * e)

        slope = (move(step) - move(-step)) / (2 * step)
        assert np.isclose(float(np.sum(f64(got[i]) * e)), slope, rtol=1e-3, atol=1e-6), f"gradient {i} against differences"


def _all_calls(blk):
    qa, sa, t, low, qkv, out = blk.forward()
    rows = tp.tp_rmsnorm_rotate(blk.x, blk.gamma, out_kind="bf16")
    return (qa, sa, t, low, qkv, out, rows) + blk.backward(qa, sa, t, low, qkv)


def _equal(got, want, what):
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), f"{what}: output {i}"


def test_side_streams_give_the_same_bytes():
    d = dev()
    announce("block on side streams")
    blk = Block(50, 512, 4, 2, 32, 8, seed=3, d=d)
    want = [v.clone() for v in _all_calls(blk)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _all_calls(blk)
    side.synchronize()
    _equal(got, want, "current stream")
    # the stream named in the call: the outputs and workspaces belong to it
    qa, sa, t = tp.tp_rmsnorm_rotate(blk.x, blk.gamma, eps=EPS, residual=blk.res, stream=side)
    low = tp.tp_lora_down_prequantized(qa, sa, blk.a, stream=side)
    q, k = tp.tp_qk_norm_rope(want[4][:, :blk.cq], want[4][:, blk.cq:blk.ck], stream=side, **blk.rope())
    grads = tp.tp_lora_grad_prequantized(want[-1], qa, sa, low, blk.b, ALPHA, stream=side)
    side.synchronize()
    _equal((qa, sa, t, low), want[:4], "named stream")
    _equal((q, k), (want[5][:, :blk.cq], want[5][:, blk.cq:blk.ck]), "named stream rope")
    _equal(grads[:2], want[7:9], "named stream gradients")


def test_two_streams_at_once():
    """Two blocks at the same time, each with outputs and workspaces of its own."""
    d = dev()
    announce("two blocks at once")
    blks = [Block(300, 1024, 4, 2, 64, 16, seed=s, d=d) for s in (5, 6)]
    want = [[v.clone() for v in _all_calls(b)] for b in blks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blks]
    got = [None, None]
    for _ in range(3):
        for i, (b, s) in enumerate(zip(blks, streams)):
            with torch.cuda.stream(s):
                got[i] = _all_calls(b)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        _equal(g, w, "two streams")


def test_graph_replays_match_eager():
    d = dev()
    announce("block captured and replayed")
    blk = Block(40, 768, 4, 2, 32, 12, seed=7, d=d)
    _all_calls(blk)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all_calls(blk)
    gen = torch.Generator(device=d)
    for rep in range(4):
        gen.manual_seed(50 + rep)
        blk.x.copy_(torch.randn(blk.x.shape, device=d, generator=gen))
        blk.grad.copy_(torch.randn(blk.grad.shape, device=d, generator=gen))
        torch.cuda.synchronize()
        want = [v.clone() for v in _all_calls(blk)]
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _equal(out, want, f"replay {rep}")
    del graph


# ------------------------------------------------- past 2^31 elements and bytes
def _far_rows(m):
    return np.unique(np.concatenate([np.arange(3), np.arange(m - 3, m), [m // 2, m // 3]]))


def test_norm_of_more_than_2_31_elements():
    d = dev()
    m, k = 530000, 4096
    announce("tp_rmsnorm_rotate", m, k)
    g = torch.Generator(device=d).manual_seed(1)
    x = torch.empty((m, k), dtype=BF16, device=d).normal_(generator=g)
    q, s = tp.tp_rmsnorm_rotate(x, None, eps=EPS)
    sel = torch.from_numpy(_far_rows(m)).to(d)
    rq, rs = oracle.quantize_activations_int8(oracle.rmsnorm(f64(x[sel]), None, EPS))
    assert np.array_equal(host(q[sel]), rq) and np.array_equal(host(s[sel]), rs)
    # the side path on those codes
    a = torch.randn((8, k), device=d, generator=g).to(BF16)
    t = tp.tp_lora_down_prequantized(q, s, a)
    mag = (np.abs(rq.astype(np.float64)) * rs.astype(np.float64)[:, None]) @ np.abs(f64(a)).T
    B.assert_sum(f64(t[sel])[:, :8], oracle.lora_down_codes(rq, rs, f64(a)), mag, k + 32, "T")
    # gradients, of dy = t
    dx, dgamma = tp.tp_rmsnorm_rotate_backward(x, x, None, eps=EPS, want_dgamma=False)
    x64 = f64(x[sel])
    want, bound, _, _ = B.norm_backward(x64, x64, None, EPS, None, True, 0)
    B.assert_close(f64(dx[sel]), want, bound, True, "dx")


def test_rope_of_more_than_2_31_elements():
    d = dev()
    m, heads, hd = 300000, 60, 128
    announce("tp_qk_norm_rope", m, heads, hd)
    g = torch.Generator(device=d).manual_seed(2)
    x = torch.empty((m, heads * hd), dtype=BF16, device=d).normal_(generator=g)
    pos = torch.arange(m, dtype=torch.int32, device=d)
    freq = (10000.0 ** (-torch.arange(64, device=d, dtype=torch.float64) / 64)).float()
    gamma = torch.ones((hd,), device=d)
    sel = torch.from_numpy(_far_rows(m)).to(d)
    keep = f64(x[sel])
    cut = 40 * hd
    q, k = tp.tp_qk_norm_rope(x[:, :cut], x[:, cut:], hd, pos, freq, q_gamma=gamma, k_gamma=gamma, q_out=x[:, :cut],
                              k_out=x[:, cut:])
    want, bound = B.rope_forward(keep, hd, host(pos[sel])[:, None], host(freq), [0] * 64, False, np.ones(hd), 1e-6)
    B.assert_close(f64(x[sel]), want, bound, True, "out")


def test_side_gradients_of_more_than_2_31_elements():
    d = dev()
    m, n, k, r = 270000, 8192, 256, 4
    announce("tp_lora_grad_prequantized", m, n, k, r)
    g = torch.Generator(device=d).manual_seed(3)
    dy = torch.empty((m, n), dtype=BF16, device=d).normal_(generator=g)
    qa = torch.randint(-127, 128, (m, k), dtype=torch.int8, device=d, generator=g)
    sa = torch.rand((m,), device=d, generator=g) + 0.5
    t = torch.zeros((m, 64), device=d)
    t[:, :r].normal_(generator=g)
    b = torch.zeros((n, 8), dtype=BF16, device=d)
    b[:, :r].normal_(generator=g)
    b = b[:, :r]
    da, db, dt = tp.tp_lora_grad_prequantized(dy, qa, sa, t, b, 1.0)
    sel = torch.from_numpy(_far_rows(m)).to(d)
    y64, b64 = f64(dy[sel]), f64(b)
    B.assert_sum(f64(dt[sel])[:, :r], y64 @ b64, np.abs(y64) @ np.abs(b64), n + 64, "dT")
    cols = torch.tensor([0, 1, n // 2, n - 1], device=d)
    yc, t64 = f64(dy[:, cols]), f64(t[:, :r])
    B.assert_sum(f64(db)[host(cols)], yc.T @ t64, np.abs(yc).T @ np.abs(t64), 3 * m, "dB")
    qc, dt64 = f64(qa[:, cols % k]) * f64(sa)[:, None], f64(dt)[:, :r]
    B.assert_sum(f64(da)[:, host(cols % k)], dt64.T @ qc, np.abs(dt64).T @ np.abs(qc), 3 * m, "dA")


def _every_argument(blk):
    """Each call with all its arguments given by name, outputs and workspaces
    too: (function, inputs, a maker of its output arguments)."""
    d = blk.x.device
    m, k, n, r, hd = blk.m, blk.k, blk.n, blk.r, blk.hd
    qa, sa, t, low, qkv, _ = blk.forward()
    f = lambda *shape: torch.full(shape, 7.0, device=d)  # noqa: E731
    b = lambda *shape: torch.full(shape, 7.0, dtype=BF16, device=d)  # noqa: E731
    ws = lambda size: torch.empty((max(size, 16),), dtype=torch.uint8, device=d)  # noqa: E731
    q, kk, dq, dk = (v[:, lo:hi] for v in (qkv, blk.grad) for lo, hi in ((0, blk.cq), (blk.cq, blk.ck)))
    rope = dict(blk.rope(), layout="halves")
    return [
        (tp.tp_rmsnorm_rotate, dict(x=blk.x, gamma=blk.gamma, eps=1e-3, residual=blk.res, rotate=False, out_kind="i8"),
         lambda: dict(out=torch.empty((m, k), dtype=torch.int8, device=d), scales=f(m), sum_out=b(m, k))),
        (tp.tp_rmsnorm_rotate_backward, dict(dy=blk.x, t=t, gamma=blk.gamma, eps=1e-3, dsum=blk.dsum, rotate=False,
                                             dx_dtype=BF16, want_dgamma=True),
         lambda: dict(dx=b(m, k), dgamma=f(k), workspace=ws(tp.tp_rmsnorm_backward_workspace_size(m, k)))),
        (tp.tp_lora_down_prequantized, dict(qa=qa, sa=sa, lora_a=blk.a),
         lambda: dict(t=f(m, 64), workspace=ws(tp.tp_lora_down_prequantized_workspace_size(m, k, r)))),
        (tp.tp_lora_grad_prequantized, dict(dy=blk.grad, qa=qa, sa=sa, t=low, lora_b=blk.b, alpha=ALPHA, rotate=True),
         lambda: dict(da=f(r, k), db=f(n, r), dt=f(m, 64), workspace=ws(tp.tp_lora_grad_workspace_size(m, n, k, r)))),
        (tp.tp_qk_norm_rope, dict(rope, q=q, k=kk, out_dtype=BF16), lambda: dict(q_out=b(m, blk.cq), k_out=b(m, blk.ck - blk.cq))),
        (tp.tp_qk_norm_rope_backward, dict(rope, dq_out=dq, dk_out=dk, q=q, k=kk, dx_dtype=BF16, want_dgamma=True),
         lambda: dict(dq=b(m, blk.cq), dk=b(m, blk.ck - blk.cq), dq_gamma=f(hd), dk_gamma=f(hd),
                      workspace=ws(tp.tp_qk_norm_rope_workspace_size(m, blk.hq, blk.hk, hd)))),
    ]


def test_every_argument_on_another_stream_or_device(monkeypatch):
    """A call that moves to a named stream, or to its tensors' device, passes
    all its arguments on: the same bytes, in the outputs that it was given."""
    d = dev()
    announce("every argument, moved calls")
    from int4_quantized_gemm_amd import block_ops
    blk = Block(33, 512, 4, 2, 32, 8, seed=11, d=d)
    side = torch.cuda.Stream()
    for fn, inputs, outputs in _every_argument(blk):
        want = [v.clone() for v in fn(**inputs)] if fn is not tp.tp_lora_down_prequantized else [fn(**inputs).clone()]
        for how in ("stream", "device"):
            outs = outputs()
            torch.cuda.synchronize()
            if how == "stream":
                got = fn(**inputs, **outs, stream=side)
            else:
                real, first = block_ops._current_device, []
                monkeypatch.setattr(block_ops, "_current_device",
                                    lambda: real() if first else first.append(1) or real() + 1)
                got = fn(**inputs, **outs)
                monkeypatch.setattr(block_ops, "_current_device", real)
                assert first
            side.synchronize()
            got = list(got) if isinstance(got, tuple) else [got]
            _equal(got, want, f"{fn.__name__} {how}")
            given = {v.data_ptr() for name, v in outs.items() if name != "workspace"}
            assert {v.data_ptr() for v in got} == given, f"{fn.__name__}: outputs of its own"


def test_tensors_of_the_host_or_wrong_shape_are_refused():
    d = dev()
    blk = Block(8, 256, 2, 1, 32, 8, seed=12, d=d)
    qa, sa, t, low, qkv, _ = blk.forward()
    with pytest.raises(ValueError, match="gamma must be a tensor on"):
        tp.tp_rmsnorm_rotate(blk.x, blk.gamma.cpu())
    with pytest.raises(ValueError, match="residual must have shape"):
        tp.tp_rmsnorm_rotate(blk.x, blk.gamma, residual=blk.res[:4])
    with pytest.raises(TypeError, match="out must be"):
        tp.tp_rmsnorm_rotate(blk.x, blk.gamma, out=torch.empty((8, 256), device=d))
    with pytest.raises(ValueError, match="unit stride"):
        tp.tp_rmsnorm_rotate(blk.x.t().contiguous().t(), blk.gamma)
    with pytest.raises(ValueError, match="contiguous vector"):
        tp.tp_lora_down_prequantized(qa, sa[:4], blk.a)
    with pytest.raises(ValueError, match="lora_b must have shape"):
        tp.tp_lora_grad_prequantized(blk.grad, qa, sa, low, blk.b[:-1], 1.0)
    with pytest.raises(ValueError, match="multiple of 48"):
        tp.tp_qk_norm_rope(qkv[:, :64], qkv[:, 64:96], 48)
    with pytest.raises(ValueError, match="pair_axis must have 16 entries"):
        tp.tp_qk_norm_rope(qkv[:, :64], qkv[:, 64:96], 32, blk.pos, blk.freq, [0] * 4)
    with pytest.raises(ValueError, match="q is needed"):
        tp.tp_qk_norm_rope_backward(qkv[:, :64], qkv[:, 64:96], None, None, 32, q_gamma=blk.qg)
    with pytest.raises(tp.TPError, match="workspace"):
        tp.tp_lora_down_prequantized(qa, sa, blk.a, workspace=torch.empty((16,), dtype=torch.uint8, device=d))
