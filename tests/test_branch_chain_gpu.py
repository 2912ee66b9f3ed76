"""Dropout, layer norm, e4m3 quantizers and products used together, as a block
uses them around a projection: the branch dropped and added to the stream, layer
norm to e4m3 codes, the product with frozen-scale weights, dropout and residual
behind it; and the way back to the stream's, the branch's, the weight's and the
norm weights' gradients. Then the same calls on other streams, in captured
graphs, with empty operands, and on buffers past 2^31 elements."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests import branch_bounds as R
from tests.gpu_util import announce, dev, f64, host, sample_rows

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS, P = 1e-5, 0.1


class Branch:
    """x the branch's output, res the stream, w [n, k] a projection, by blocks in
    the rotated domain."""

    def __init__(self, m, k, n, seed, d):
        rng = np.random.default_rng(seed)
        draw = lambda shape, s=1.0: torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(s))  # noqa: E731
        self.m, self.k, self.n = m, k, n
        self.x, self.res = draw((m, k)).to(d), draw((m, k), 2.0).to(BF16).to(d)
        self.gamma, self.beta = (1.0 + draw((k,), 0.1)).to(BF16).to(d), draw((k,), 0.1).to(BF16).to(d)
        self.w, self.ws, self.wt, self.wst = tp.tp_quantize_fp8(draw((n, k), 0.02).to(d), block_rows=128, rotate=True, want="both")
        # rows of 16-byte pitches whatever n
        wide = lambda t: torch.nn.functional.pad(t, (0, -n % 4)).to(d)[:, :n]  # noqa: E731
        self.res2, self.grad = wide(draw((m, n))), wide(draw((m, n), 0.02))
        self.dsum = draw((m, k), 0.02).to(BF16).to(d)
        self.rng = torch.tensor([77, 5], dtype=torch.int64, device=d)
        self.rng2 = torch.tensor([77, 6], dtype=torch.int64, device=d)

    def forward(self):
        h, hs, t = tp.tp_layernorm_rotate(self.x, self.gamma, self.beta, eps=EPS, residual=self.res, drop_p=P, rng=self.rng,
                                          out_kind="fp8")
        y = torch.empty((self.m, self.n + -self.n % 4), device=h.device)[:, :self.n]
        tp.tp_qgemm_fp8(h, hs, self.w, self.ws, out=y)
        return h, hs, t, y, tp.tp_dropout(y, P, self.rng2, residual=self.res2)

    def backward(self, h, hs, t):
        dy = tp.tp_dropout(self.grad, P, self.rng2)
        g, gs, gt, gst = tp.tp_quantize_fp8(dy, want="both")
        dh = tp.tp_qgemm_fp8(g, gs, self.wt, self.wst)  # [m, k], in the rotated domain
        # h by columns for the weight's gradient: made again from the stream
        rows = tp.tp_layernorm_rotate(t, self.gamma, self.beta, eps=EPS, out_kind="bf16")
        ht, hst = tp.tp_quantize_fp8(rows, want="cols")
        dw = tp.tp_qgemm_fp8(gt, gst, ht, hst, b_block_rows=1)
        dx, branch, dgamma, dbeta = tp.tp_layernorm_rotate_backward(dh, t, self.gamma, eps=EPS, dsum=self.dsum, drop_p=P,
                                                                    rng=self.rng)
        return dy, g, gs, gt, gst, dh, rows, ht, hst, dw, dx, branch, dgamma, dbeta


def _codes(t):
    return host(t.view(torch.uint8))


@pytest.mark.parametrize("m,k,n", [(64, 1024, 640), (37, 768, 300), (300, 4352, 1163)])
def test_branch_forward_and_gradients(m, k, n):
    d = dev()
    announce("branch forward and backward", m, k, n)
    b = Branch(m, k, n, seed=m, d=d)
    h, hs, t, y, out = b.forward()
    seed, off = 77, 5
    keep, keep2 = oracle.drop_keep(seed, off, m, k, P), oracle.drop_keep(seed, off + 1, m, n, P)
    t64 = oracle.stream_sum(oracle.dropped(f64(b.x), keep, P), f64(b.res), True)
    assert np.array_equal(f64(t), t64)
    q, s = oracle.quantize_fp8_rows(oracle.rotate_groups(oracle.layernorm(t64, f64(b.gamma), f64(b.beta), EPS)))
    assert np.array_equal(_codes(h), q) and np.array_equal(host(hs), s)
    want, mag = oracle.qgemm_fp8(q, s, _codes(b.w), host(b.ws))
    B.assert_close(f64(y), want, R.product(mag, k, False), False, "y")
    assert np.array_equal(f64(out), oracle.dropout(f64(y), keep2, P, f64(b.res2), False))

    dy, g, gs, gt, gst, dh, rows, ht, hst, dw, dx, branch, dgamma, dbeta = b.backward(h, hs, t)
    assert np.array_equal(f64(dy), oracle.dropout(f64(b.grad), keep2, P, None, False))
    q, s = oracle.quantize_fp8_rows(f64(dy))
    qt, st = oracle.quantize_fp8_cols(f64(dy))
    assert np.array_equal(_codes(g), q) and np.array_equal(host(gs), s)
    assert np.array_equal(_codes(gt), qt) and np.array_equal(host(gst), st)
    want, mag = oracle.qgemm_fp8(q, s, _codes(b.wt), host(b.wst))
    B.assert_close(f64(dh), want, R.product(mag, q.shape[1], False), False, "dh")
    want, mag = oracle.qgemm_fp8(qt, st, _codes(ht), host(hst), 1)
    B.assert_close(f64(dw), want, R.product(mag, qt.shape[1], False), False, "dw")
    want = R.layernorm_backward(f64(dh), t64, f64(b.gamma), EPS, f64(b.dsum), True, m + 40)
    B.assert_close(f64(dx), want[0], want[1], True, "dx")
    B.assert_close(f64(dgamma), want[2], want[3], False, "dgamma")
    B.assert_close(f64(dbeta), want[4], want[5], False, "dbeta")

    # against differences of <dy as coded, h' w^T> + <dsum, t>, the function that
    # these gradients belong to, along random directions
    dq = np.repeat(s.T, 128, axis=1) * oracle.e4m3_value(q)
    wfull = np.repeat(np.repeat(host(b.ws).astype(np.float64), 128, axis=0)[:n], 128, axis=1) * oracle.e4m3_value(_codes(b.w))
    back = dq[:, :n] @ wfull

    def loss(x, gamma, beta):
        tt = np.where(keep, x * float(oracle.drop_factor(P)), 0.0) + f64(b.res)
        return float(np.sum(back * oracle.rotate_groups(oracle.layernorm(tt, gamma, beta, EPS))) + np.sum(f64(b.dsum) * tt))

    rng = np.random.default_rng(2)
    at = [f64(b.x), f64(b.gamma), f64(b.beta)]
    for i, got in ((0, branch), (1, dgamma), (2, dbeta)):
        e = rng.standard_normal(at[i].shape)
        step = 1e-4 / np.linalg.norm(e)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * e, at[i] - step * e
        slope = (loss(*up) - loss(*down)) / (2 * step)
        # the stream is rounded to bf16 in the kernel's forward and not here (2^-8
        # of its values, so of n), the branch's gradient is bf16: two roundings of
        # 2^-8 against the terms' norm, as the directions are random signs
        room = 4 * 2 * B.HALF_BF16 * float(np.linalg.norm(f64(got) * e))
        assert abs(float(np.sum(f64(got) * e)) - slope) <= room, f"gradient {i} against differences"


def _all_calls(b):
    h, hs, t, y, out = b.forward()
    return (h, hs, t, y, out) + b.backward(h, hs, t)


def _equal(got, want, what):
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), f"{what}: output {i}"


def test_side_streams_give_the_same_bytes():
    """On another stream, and on two at once, each with its own allocations (m and
    k take the split product and its workspace)."""
    d = dev()
    announce("branch on side streams")
    b = Branch(300, 4352, 640, seed=3, d=d)
    assert tp.tp_qgemm_fp8_workspace_size(300, 640, 4352) > 0, "the product is meant to split k"
    want = _all_calls(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(_all_calls(b))
    for s in streams:
        s.synchronize()
    for g in got:
        _equal(g, want, "side stream")
    y = torch.zeros_like(want[3])
    tp.tp_qgemm_fp8(want[0], want[1], b.w, b.ws, out=y, stream=streams[0])
    streams[0].synchronize()
    _equal((y,), (want[3],), "stream argument")


def test_graph_replays_draw_new_masks():
    """Captured once, replayed with new seeds, offsets and inputs, eager work in
    between; two graphs of one pool do not disturb each other."""
    d = dev()
    announce("branch in graphs")
    b, c = Branch(130, 1280, 384, seed=4, d=d), Branch(3, 4352, 300, seed=5, d=d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_calls(b), _all_calls(c)
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g, blk in zip(graphs, (b, c)):
        with torch.cuda.graph(g, stream=side):
            outs.append(_all_calls(blk))
    seen = []
    for i in range(4):
        for blk in (b, c):
            blk.rng[1] = 1000 + 17 * i
            blk.rng2[0] = 5 * i
            blk.x.normal_()
        graphs[i & 1].replay()
        graphs[1 - (i & 1)].replay()
        torch.cuda.synchronize()
        for blk, out in zip((b, c), outs):
            _equal(out, _all_calls(blk), f"replay {i}")
        seen.append(outs[0][4].clone())
        torch.cuda.synchronize()
    assert not any(torch.equal(seen[i], seen[j]) for i in range(4) for j in range(i))


def test_empty_operands():
    d = dev()
    announce("empty operands")
    e = torch.zeros((0, 512), device=d)
    rng = torch.tensor([1, 2], dtype=torch.int64, device=d)
    assert tp.tp_dropout(e, 0.5, rng).shape == (0, 512) and tp.tp_dropout(torch.zeros((4, 0), device=d), 0.5, rng).shape == (4, 0)
    for kind in ("i8", "bf16", "fp8"):
        got = tp.tp_layernorm_rotate(e, residual=e, drop_p=0.5, rng=rng, out_kind=kind)
        assert got[0].shape == (0, 512) and got[-1].shape == (0, 512)
    q, s, qt, st = tp.tp_quantize_fp8(e, want="both")
    assert q.shape == (0, 512) and s.shape == (4, 0) and qt.shape == (512, 0) and st.shape == (0, 512)
    w, ws = tp.tp_quantize_fp8(torch.ones((3, 512), device=d), block_rows=128)
    assert tp.tp_qgemm_fp8(q, s, w, ws).shape == (0, 3)
    a, sa = tp.tp_quantize_fp8(torch.ones((3, 512), device=d))
    n0 = torch.zeros((0, 512), device=d).to(F8)
    assert tp.tp_qgemm_fp8(a, sa, n0, torch.zeros((0, 4), device=d)).shape == (3, 0)


# ------------------------------------------------------------ past 2^31 elements
def _noise(m, k, d, seed):
    g = torch.Generator(device=d).manual_seed(seed)
    x = torch.empty((m, k), dtype=BF16, device=d)
    for r in range(0, m, 8192):
        x[r:r + 8192].normal_(generator=g)
    return x


def test_rows_past_2g_elements():
    d = dev()
    m, k = 140001, 16384
    announce("rows past 2^31 elements", m, k)
    assert m * k > 2 ** 31
    x = _noise(m, k, d, 1)
    rows = sample_rows(m, 4, 1)
    rows = np.array([r for r in rows if r < 2 or r > m - 3 or r > 131072][-6:])
    x64 = f64(x[torch.from_numpy(rows).to(d)])
    rng = torch.tensor([9, 8], dtype=torch.int64, device=d)
    keep = oracle.drop_keep(9, 8, m, k, 0.1, rows=rows)
    pick = lambda t: t[torch.from_numpy(rows).to(d)]  # noqa: E731
    y = tp.tp_dropout(x, 0.1, rng)
    assert np.array_equal(f64(pick(y)), oracle.dropout(x64, keep, 0.1, None, True))
    q, s, t = tp.tp_layernorm_rotate(x, eps=EPS, residual=y, drop_p=0.1, rng=rng, out_kind="fp8", sum_out=y)
    t64 = oracle.stream_sum(oracle.dropped(x64, keep, 0.1), oracle.dropout(x64, keep, 0.1, None, True), True)
    assert np.array_equal(f64(pick(t)), t64)
    wq, ws = oracle.quantize_fp8_rows(oracle.rotate_groups(oracle.layernorm(t64, None, None, EPS)))
    assert np.array_equal(_codes(pick(q)), wq) and np.array_equal(host(s[:, torch.from_numpy(rows).to(d)]), ws)
    del q, s
    dx, branch, dgamma, _ = tp.tp_layernorm_rotate_backward(x, t, eps=EPS, drop_p=0.1, rng=rng, rotate=False, want_dbeta=False)
    want = R.layernorm_backward(x64, t64, None, EPS, None, False, 1)
    B.assert_close(f64(pick(dx)), want[0], want[1], True, "dx")
    factor = float(oracle.drop_factor(0.1))
    B.assert_close(f64(pick(branch)), np.where(keep, want[0] * factor, 0),
                   np.where(keep, (want[1] + B.U * np.abs(want[0])) * factor, 0), True, "dbranch")


@pytest.mark.parametrize("k", [1024, 4352])
def test_more_rows_than_blocks_of_a_launch(k):
    """More rows than one launch takes blocks (2^21): the second launch's rows, and
    the last of the first's."""
    d = dev()
    m = 2 ** 21 + 77
    announce("more rows than blocks", m, k)
    x = _noise(m, k, d, 3)
    rows = np.array([0, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 1, m - 1])
    at = torch.from_numpy(rows).to(d)
    x64 = f64(x[at])
    q, s = tp.tp_layernorm_rotate(x, eps=EPS, out_kind="fp8")
    wq, ws = oracle.quantize_fp8_rows(oracle.rotate_groups(oracle.layernorm(x64, None, None, EPS)))
    assert np.array_equal(_codes(q.view(torch.uint8)[at]), wq) and np.array_equal(host(s[:, at]), ws)
    del q, s
    dx, _, _, dbeta = tp.tp_layernorm_rotate_backward(x, x, eps=EPS, rotate=False, want_dgamma=False)
    want = R.layernorm_backward(x64, x64, None, EPS, None, False, 1)
    B.assert_close(f64(dx[at]), want[0], want[1], True, "dx")
    total = sum(x[r:r + 65536].double().sum(dim=0) for r in range(0, m, 65536))
    size = sum(x[r:r + 65536].abs().double().sum(dim=0) for r in range(0, m, 65536))
    # a thread adds up to m / 512 rows one by one, then 512 partial rows by 16s
    room = (m / 512 + 80) * B.U * f64(size.float()) * 1.01
    assert np.all(np.abs(f64(dbeta) - total.cpu().numpy()) <= room)


def test_codes_past_2g_elements():
    d = dev()
    m, k = 140001, 16384
    announce("codes past 2^31 elements", m, k)
    x = _noise(m, k, d, 2)
    q, s, qt, st = tp.tp_quantize_fp8(x, want="both")
    for r in (0, m // 2, m - 1):
        wq, ws = oracle.quantize_fp8_rows(f64(x[r:r + 1]))
        assert np.array_equal(_codes(q[r:r + 1]), wq) and np.array_equal(host(s[:, r:r + 1]), ws)
    for c in (0, k - 1):
        wq, ws = oracle.quantize_fp8_cols(f64(x[:, c:c + 1]))
        assert np.array_equal(_codes(qt[c:c + 1]), wq) and np.array_equal(host(st[:, c:c + 1]), ws)


def test_products_past_2g_elements():
    """Rows of a and of b, and elements of c, past 2^31; whole numbers, exact."""
    d = dev()
    m, n, k = 66000, 32900, 128
    announce("product past 2^31 elements", m, n, k)
    assert m * n > 2 ** 31
    g = torch.Generator(device=d).manual_seed(6)
    a, b = (torch.randint(-8, 9, (r, k), generator=g, device=d).float() for r in (m, n))
    sa, sb = torch.ones((1, m), device=d), torch.ones((-(-n // 128), 1), device=d)
    for dtype in (BF16, F32):
        c = tp.tp_qgemm_fp8(a.to(F8), sa, b.to(F8), sb, out_dtype=dtype)
        for r in (slice(0, 256), slice(m - 300, m)):
            assert torch.equal(c[r], (a[r] @ b.t().contiguous()).to(dtype)), dtype
        del c


def test_long_sums_past_2g_codes():
    """Operands of more than 2^31 codes: k near its largest."""
    d = dev()
    m, n, k = 300, 5, 2 ** 24 - 128
    announce("product of long rows", m, n, k)
    assert m * k > 2 ** 31
    g = torch.Generator(device=d).manual_seed(7)
    a = torch.zeros((m, k), dtype=torch.uint8, device=d)
    b = torch.randint(-8, 9, (n, k), generator=g, device=d).to(F8)
    where = torch.randint(0, k, (64,), generator=g, device=d)
    a[:, where] = 0x38  # 1
    a[m - 1, k - 1] = 0x40  # 2
    sa, sb = torch.ones((k // 128, m), device=d), torch.ones((1, k // 128), device=d)
    cols = torch.unique(torch.cat([where, torch.tensor([k - 1], device=d)]))
    some = lambda t: t.view(torch.uint8)[:, cols].contiguous().view(F8).float()  # noqa: E731
    want, a = some(a) @ some(b).t().contiguous(), a.view(F8)
    for dtype in (F32, BF16):
        assert torch.equal(tp.tp_qgemm_fp8(a, sa, b, sb, out_dtype=dtype), want.to(dtype))
