"""The norms at the far ends of fp32: rows whose elements are finite but whose
sums, factors or products of factors would leave fp32's range if they were taken
in the wrong order. The bounds are those of ordinary rows: nothing is allowed for
the size of the values."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests import block_bounds as B
from tests.gpu_util import announce, dev, f64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _normal(shape, seed, dtype=F32):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def _large_rows(k, dtype):
    """Rows up to fp32's (bf16's) largest values: a constant one, whose rotated
    groups are 256 times an element before the row factor, one whose groups all
    reach the end of the range, one with a single large element, alternating
    signs, and ordinary rows between them."""
    x = _normal((9, k), k).numpy()
    x[0] = 3e36
    x[2] = np.clip(x[2], -3.3, 3.3) * np.float32(1e38)
    x[3] = 1.0
    x[3, k // 2 + 5] = -3.3e38
    x[5] = 3.3e38
    x[6] = np.where(np.arange(k) % 2 == 0, 2e38, -2e38)
    x[7] *= np.float32(1e35)
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("k", [256, 768, 1024, 4352])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rotate", [True, False])
def test_norm_rows_at_the_end_of_the_range(k, dtype, rotate):
    d = dev()
    announce("tp_rmsnorm_rotate large rows", k, dtype, rotate)
    x = _large_rows(k, dtype)
    # (t gamma itself has to stay in fp32)
    gamma = (0.75 + 0.05 * _normal((k,), k + 1)).clamp(0.5, 1.0)
    for gam in (None, gamma, gamma.to(BF16)):
        g64 = None if gam is None else f64(gam)
        rows = tp.tp_rmsnorm_rotate(x.to(d), None if gam is None else gam.to(d), out_kind="bf16", rotate=rotate)
        want, bound = B.norm_rows(f64(x), g64, 1e-6, rotate)
        B.assert_close(f64(rows), want, bound, True, "rows")
    # as the new stream: the sum, and the rows of it
    res = torch.zeros_like(x)
    rows, t = tp.tp_rmsnorm_rotate(x.to(d), gamma.to(d), residual=res.to(d), out_kind="bf16", rotate=rotate)
    want, bound = B.norm_rows(f64(x), f64(gamma), 1e-6, rotate)
    B.assert_close(f64(rows), want, bound, True, "rows of the stream")
    assert torch.equal(t.cpu(), x)


@pytest.mark.parametrize("k", [256, 512, 768, 1024, 4352])
@pytest.mark.parametrize("rotate", [True, False])
def test_rows_beside_large_and_non_finite_rows_keep_their_bytes(k, rotate):
    """Rows that share a wave or a block with rows at the end of the range, or
    with infinities and NaN, are the rows that they are alone."""
    d = dev()
    announce("tp_rmsnorm_rotate beside large rows", k, rotate)
    x = _normal((41, k), k + 9)
    gamma = (1.0 + 0.1 * _normal((k,), k + 1)).to(d)
    want = tp.tp_rmsnorm_rotate(x.to(d), gamma, out_kind="bf16", rotate=rotate)
    bad = x.clone()
    bad[1], bad[6, 3], bad[11, 5], bad[16, 7], bad[22] = 3e38, float("inf"), float("nan"), float("-inf"), -2e37
    got = tp.tp_rmsnorm_rotate(bad.to(d), gamma, out_kind="bf16", rotate=rotate)
    keep = [i for i in range(41) if i not in (1, 6, 11, 16, 22)]
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))


def _scaled_rows(k, seed):
    """Rows of every size: with a mean square from far below eps to 2^250."""
    t = _normal((10, k), seed).numpy()
    for i, s in enumerate((1.0, 1e-25, 1e-12, 1e6, 1e18, 1e21, 1e23, 1e30, 1e36, 1.0)):
        t[i] *= np.float32(s)
    t[8] = np.clip(t[8], -3e36, 3e36)
    return torch.from_numpy(t)


@pytest.mark.parametrize("m,k", [(10, 256), (10, 1024), (10, 4352)])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_norm_backward_of_rows_of_any_size(m, k, rotate, eps):
    """dx row by row. dgamma too: column sums over rows whose factors are as far
    apart as 1e25 and 1e-36, which weigh the same in it."""
    d = dev()
    announce("tp_rmsnorm_rotate_backward rows of any size", m, k, rotate, eps)
    t, dy, gamma = _scaled_rows(k, k), _normal((m, k), k + 1) * 1e-3, 1.0 + 0.1 * _normal((k,), k + 2)
    for gam in (None, gamma):
        g64 = None if gam is None else f64(gam)
        dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None if gam is None else gam.to(d), eps=eps,
                                               rotate=rotate)
        want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), g64, eps, None, rotate, m + 64)
        B.assert_close(f64(dx), want, bound, False, "dx")
        B.assert_close(f64(dg), wdg, bdg, False, "dgamma")
        # a gradient of the stream beside it
        ds = _normal((m, k), k + 3)
        dx, _ = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None if gam is None else gam.to(d), eps=eps,
                                              dsum=ds.to(d), rotate=rotate)
        want, bound, _, _ = B.norm_backward(f64(dy), f64(t), g64, eps, f64(ds), rotate, m + 64)
        B.assert_close(f64(dx), want, bound, False, "dx with dsum")


@pytest.mark.parametrize("m,k", [(10, 768), (10, 4352)])
def test_norm_backward_of_large_rows_and_gradients(m, k):
    """Products of large rows with ordinary and with large gradients: the sum of
    gamma g t is past fp32 where dx is not."""
    d = dev()
    announce("tp_rmsnorm_rotate_backward large rows and gradients", m, k)
    t, dy = _scaled_rows(k, k + 4), _normal((m, k), k + 5)
    dy[5:] *= 1e6
    dx, dg = tp.tp_rmsnorm_rotate_backward(dy.to(d), t.to(d), None)
    want, bound, wdg, bdg = B.norm_backward(f64(dy), f64(t), None, 1e-6, None, True, m + 64)
    B.assert_close(f64(dx), want, bound, False, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")


@pytest.mark.parametrize("hd,pairs,layout", [(64, 32, "interleaved"), (80, 16, "halves"), (256, 128, "halves")])
def test_rope_backward_of_large_and_small_heads(hd, pairs, layout):
    """Heads whose squares add up just inside fp32, with small gradients: the
    cube of the head's factor is far below fp32's range, dx is not."""
    d = dev()
    announce("tp_qk_norm_rope_backward large heads", hd, pairs, layout)
    m, heads = 6, 5
    w = heads * hd
    x, dy = _normal((m, w), hd).numpy(), _normal((m, w), hd + 1) * 1e-6
    for i, s in enumerate((1.0, 1e12, 1e16, 6e17, 1e-12, 1.0)):
        x[i] *= np.float32(s)
    x = torch.from_numpy(x)
    rng = np.random.default_rng(hd)
    pos = torch.from_numpy(rng.integers(-50, 50, size=(m, 1)).astype(np.int32))
    freq = torch.from_numpy((100.0 ** (-np.arange(pairs) / pairs)).astype(np.float32))
    gamma = 1.0 + 0.1 * _normal((hd,), hd + 2)
    none = x[:, :0].to(d)
    dx, _, dg, _ = tp.tp_qk_norm_rope_backward(dy.to(d), none, x.to(d), none, hd, pos.to(d), freq.to(d), None, layout,
                                               gamma.to(d), eps=1e-5)
    want, bound, wdg, bdg = B.rope_backward(f64(dy), f64(x), hd, pos.numpy(), freq.numpy(), [0] * pairs,
                                            layout == "halves", f64(gamma), 1e-5, m * heads + 400)
    B.assert_close(f64(dx), want, bound, False, "dx")
    B.assert_close(f64(dg), wdg, bdg, False, "dgamma")
