"""tp_qk_norm_rope and its gradients against the fp64 oracle, inside the bounds
of the fp32 arithmetic (angles are fp64 on both sides)."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# tokens, heads of q and k, head_dim, pairs, axes: one token, shared key heads,
# no key heads, widths that leave lanes of a group idle, partial and no
# rotation, more heads than a block turns at once, more tokens than blocks
CASES = [(1, 1, 1, 8, 4, 1), (1, 32, 8, 128, 64, 1), (3, 5, 1, 80, 40, 2), (7, 2, 2, 64, 16, 3), (33, 7, 0, 96, 48, 4),
         (17, 0, 3, 256, 128, 2), (5, 40, 40, 128, 32, 3), (2, 3, 2, 16, 0, 1), (130, 6, 2, 72, 36, 2),
         (1100, 9, 4, 24, 8, 1)]


def _draw(shape, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(scale)).to(dtype)


def _plan(m, pairs, axes, seed, far):
    rng = np.random.default_rng(seed)
    pos = rng.integers(-far, far + 1, size=(m, axes)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    axis = sorted(rng.integers(0, axes, size=pairs).tolist())
    return torch.from_numpy(pos), torch.from_numpy(freq), axis


def _gamma(d, dtype, seed):
    return (1.0 + _draw((d,), F32, seed, 0.1)).to(dtype)


def _adds(m, heads):
    return (heads + 7) // 8 * ((m + 511) // 512) + 400


@pytest.mark.parametrize("m,hq,hk,d,pairs,axes", CASES)
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("xdt,odt", [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)])
def test_forward(m, hq, hk, d, pairs, axes, layout, xdt, odt):
    dv = dev()
    announce("tp_qk_norm_rope", m, hq, hk, d, pairs, axes, layout, xdt, odt)
    qk = _draw((m, (hq + hk) * d), xdt, seed=m + d, scale=1.5)
    pos, freq, axis = _plan(m, pairs, axes, seed=d, far=5000)
    qkd = qk.to(dv)
    for qg, kg in ((None, None), (_gamma(d, BF16, 1), _gamma(d, BF16, 2)), (None, _gamma(d, F32, 3))):
        on = lambda t: None if t is None else t.to(dv)  # noqa: E731
        out = tp.tp_qk_norm_rope(qkd[:, :hq * d], qkd[:, hq * d:], d, pos.to(dv), freq.to(dv) if pairs else None, axis,
                                 layout, on(qg), on(kg), eps=1e-5, out_dtype=odt)
        for x, gamma, y in ((qk[:, :hq * d], qg, out[0]), (qk[:, hq * d:], kg, out[1])):
            if x.shape[1] == 0:
                assert y.shape == (m, 0)
                continue
            want, bound = B.rope_forward(f64(x), d, pos.numpy(), freq.numpy(), axis, layout == "halves",
                                         None if gamma is None else f64(gamma), 1e-5)
            B.assert_close(f64(y), want, bound, odt == BF16, "out")


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 30])
def test_far_positions(far):
    """Angles of positions that fp32 does not hold."""
    dv = dev()
    announce("tp_qk_norm_rope far positions", far)
    m, d = 50, 64
    x = _draw((m, 2 * d), F32, seed=5)
    pos = torch.from_numpy((far - np.arange(m) * 3).astype(np.int32)[:, None] * np.array([[1, -1]], dtype=np.int32))
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    axis = [0] * 16 + [1] * 16
    q, _ = tp.tp_qk_norm_rope(x.to(dv), x[:, :0].to(dv), d, pos.to(dv), freq.to(dv), axis)
    want, bound = B.rope_forward(f64(x), d, pos.numpy(), freq.numpy(), axis, False, None, 1e-6)
    # the angle itself is an fp64 product on both sides; taken to a fraction of
    # a turn it keeps 2^-52 of its size
    bound = bound + 4 * 2.0 ** -52 * far * np.abs(f64(x)).max()
    B.assert_close(f64(q), want, bound, False, "q")


@pytest.mark.parametrize("m,hq,hk,d,pairs,axes", CASES)
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("ydt,xdt,ddt", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, BF16), (BF16, F32, F32)])
def test_backward(m, hq, hk, d, pairs, axes, layout, ydt, xdt, ddt):
    dv = dev()
    announce("tp_qk_norm_rope_backward", m, hq, hk, d, pairs, axes, layout, ydt, xdt, ddt)
    w = (hq + hk) * d
    qk, dy = _draw((m, w), xdt, seed=m + d, scale=1.5), _draw((m, w), ydt, seed=m + d + 1, scale=0.02)
    pos, freq, axis = _plan(m, pairs, axes, seed=d, far=5000)
    qkd, dyd = qk.to(dv), dy.to(dv)
    c = hq * d
    for qg, kg in ((None, None), (_gamma(d, BF16, 1), _gamma(d, BF16, 2)), (_gamma(d, F32, 3), None)):
        on = lambda t: None if t is None else t.to(dv)  # noqa: E731
        out = tp.tp_qk_norm_rope_backward(dyd[:, :c], dyd[:, c:], None if qg is None else qkd[:, :c],
                                          None if kg is None else qkd[:, c:], d, pos.to(dv),
                                          freq.to(dv) if pairs else None, axis, layout, on(qg), on(kg), eps=1e-5,
                                          dx_dtype=ddt)
        for lo, hi, gamma, dx, dg, heads in ((0, c, qg, out[0], out[2], hq), (c, w, kg, out[1], out[3], hk)):
            want, bound, wdg, bdg = B.rope_backward(f64(dy[:, lo:hi]), f64(qk[:, lo:hi]), d, pos.numpy(), freq.numpy(),
                                                    axis, layout == "halves", None if gamma is None else f64(gamma),
                                                    1e-5, _adds(m, hq + hk)) if heads else (None,) * 4
            if not heads:
                assert dx.shape == (m, 0) and (gamma is None or torch.all(dg == 0))
                continue
            B.assert_close(f64(dx), want, bound, ddt == BF16, "dx")
            assert (dg is None) == (gamma is None)
            if gamma is not None:
                B.assert_close(f64(dg), wdg, bdg, False, "dgamma")


def test_in_place_on_the_qkv_buffer():
    """q and k turned where they lie, v and what is around it untouched; then
    the gradients in place too."""
    dv = dev()
    announce("tp_qk_norm_rope in place")
    m, hq, hk, d = 37, 4, 2, 32
    w = (hq + 2 * hk) * d
    qkv = _draw((m, w), F32, seed=1).to(dv)
    pos, freq, axis = _plan(m, 16, 3, seed=2, far=50)
    how = dict(head_dim=d, positions=pos.to(dv), inv_freq=freq.to(dv), pair_axis=axis, q_gamma=_gamma(d, F32, 3).to(dv),
               k_gamma=_gamma(d, F32, 4).to(dv))
    cq, ck = hq * d, (hq + hk) * d
    want = tp.tp_qk_norm_rope(qkv[:, :cq], qkv[:, cq:ck], **how)
    buf = qkv.clone()
    tp.tp_qk_norm_rope(buf[:, :cq], buf[:, cq:ck], q_out=buf[:, :cq], k_out=buf[:, cq:ck], **how)
    assert torch.equal(buf[:, :cq], want[0]) and torch.equal(buf[:, cq:ck], want[1])
    assert torch.equal(buf[:, ck:], qkv[:, ck:])
    dy = _draw((m, w), F32, seed=6).to(dv)
    want = tp.tp_qk_norm_rope_backward(dy[:, :cq], dy[:, cq:ck], qkv[:, :cq], qkv[:, cq:ck], **how)
    buf = dy.clone()
    got = tp.tp_qk_norm_rope_backward(buf[:, :cq], buf[:, cq:ck], qkv[:, :cq], qkv[:, cq:ck], dq=buf[:, :cq],
                                      dk=buf[:, cq:ck], **how)
    assert all(torch.equal(g, x) for g, x in zip(got, want)) and torch.equal(buf[:, ck:], dy[:, ck:])
    got = tp.tp_qk_norm_rope_backward(dy[:, :cq], dy[:, cq:ck], qkv[:, :cq], qkv[:, cq:ck], want_dgamma=False, **how)
    assert got[2] is None and got[3] is None and torch.equal(got[0], want[0])
    none = tp.tp_qk_norm_rope_backward(dy[:0, :cq], dy[:0, cq:ck], qkv[:0, :cq], qkv[:0, cq:ck],
                                       **dict(how, positions=pos.to(dv)[:0]))
    assert torch.all(none[2] == 0) and torch.all(none[3] == 0) and none[0].shape == (0, cq)


def test_columns_past_the_rotation_pass_anything():
    """What is not turned is copied bit for bit, infinities and NaN too."""
    dv = dev()
    announce("tp_qk_norm_rope pass-through")
    m, d = 9, 32
    x = _draw((m, d), F32, seed=1)
    x[:, 17], x[:, 30] = float("inf"), float("nan")
    pos, freq, axis = _plan(m, 8, 1, seed=2, far=50)
    for layout in ("interleaved", "halves"):
        q, _ = tp.tp_qk_norm_rope(x.to(dv), x[:, :0].to(dv), d, pos.to(dv), freq.to(dv), axis, layout)
        assert torch.equal(q[:, 16:].cpu().view(torch.int32), x[:, 16:].contiguous().view(torch.int32))
        assert torch.all(torch.isfinite(q[:, :16]))


def test_heads_of_zeros_at_the_smallest_eps():
    dv = dev()
    announce("tp_qk_norm_rope zero heads")
    m, d = 5, 64
    x, dy = _draw((m, 3 * d), F32, seed=1), _draw((m, 3 * d), F32, seed=2, scale=0.02)
    x[3, d:2 * d] = 0.0
    pos, freq, axis = _plan(m, 32, 1, seed=3, far=50)
    g = _gamma(d, F32, 4)
    how = dict(head_dim=d, positions=pos.to(dv), inv_freq=freq.to(dv), pair_axis=axis, q_gamma=g.to(dv), eps=1e-30)
    xd, none = x.to(dv), x[:, :0].to(dv)
    for odt in (F32, BF16):
        y, _ = tp.tp_qk_norm_rope(xd, none, out_dtype=odt, **how)
        want, bound = B.rope_forward(f64(x), d, pos.numpy(), freq.numpy(), axis, False, f64(g), 1e-30)
        B.assert_close(f64(y), want, bound, odt == BF16, "out")
        assert torch.all(y[3, d:2 * d] == 0)
    dx, _, dg, _ = tp.tp_qk_norm_rope_backward(dy.to(dv), none, xd, none, **how)
    want, bound, wdg, bdg = B.rope_backward(f64(dy), f64(x), d, pos.numpy(), freq.numpy(), axis, False, f64(g), 1e-30,
                                            _adds(m, 3))
    B.assert_close(f64(dx), want, bound, False, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")
