"""The LoRA side path on 8-bit activations (tp_lora_down_prequantized) and its
gradients (tp_lora_grad_prequantized) against the fp64 oracle.

Products of codes and bf16 values are exact; an fp32 operand is three exact
bf16 parts, so a product of it counts as three terms, one of two such operands
as six, whose left-out parts are below 3 U of it. Every output is a fp32 sum
of such terms, bounded element by element; sums of one term (m, n or k of one
row) leave room for nothing but the last bits.
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


def _codes(m, k, seed):
    rng = np.random.default_rng(seed)
    qa = rng.integers(-127, 128, size=(m, k)).astype(np.int8)
    sa = rng.uniform(1e-3, 0.1, size=m).astype(np.float32)
    if m > 4:
        sa[3], qa[3] = 0.0, 0  # a row of zeros
    return torch.from_numpy(qa), torch.from_numpy(sa)


def _mat(shape, dtype, seed, scale=1.0):
    """A matrix whose row pitch is a multiple of 16 bytes, with NaN in the padding."""
    rng = np.random.default_rng(seed)
    pitch = -(-max(shape[1], 1) // 8) * 8
    full = torch.full((shape[0], pitch), float("nan"), dtype=dtype)
    full[:, :shape[1]] = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(scale)).to(dtype)
    return full


def _on(d, full, cols):
    return full.to(d)[:, :cols]


def _parts(*dtypes):
    n = sum(t == F32 for t in dtypes)
    return (1, 3, 6)[n]


@pytest.mark.parametrize("m,k,r", [(1, 256, 1), (5, 256, 16), (16, 512, 13), (17, 1280, 32), (40, 3072, 24),
                                   (257, 768, 64), (3, 12288, 8)])
@pytest.mark.parametrize("adt", [BF16, F32])
def test_down(m, k, r, adt):
    d = dev()
    announce("tp_lora_down_prequantized", m, k, r, adt)
    qa, sa = _codes(m, k, seed=m + k)
    a = _mat((r, k), adt, seed=r, scale=k ** -0.5)
    t = host(tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), _on(d, a, k))).astype(np.float64)
    x, a64 = f64(qa) * f64(sa)[:, None], f64(a[:, :k])
    B.assert_sum(t[:, :r], oracle.lora_down_codes(qa.numpy(), sa.numpy(), a64), np.abs(x) @ np.abs(a64).T,
                 k * _parts(adt) + 32, "T")
    assert np.all(t[:, r:] == 0)


def test_down_matches_the_path_on_wide_activations():
    """Codes of a real quantization: the same T as tp_lora_down on what they stand for."""
    d = dev()
    announce("tp_lora_down_prequantized against tp_lora_down")
    m, k, r = 70, 1024, 16
    x = _mat((m, k), BF16, seed=1)
    qa, sa = tp.tp_quantize_rows_int8(x.to(d))
    a = _mat((r, k), F32, seed=2, scale=k ** -0.5).to(d)
    t = tp.tp_lora_down_prequantized(qa, sa, a)
    wide = (qa.float() * sa[:, None]).contiguous()
    ref = tp.tp_lora_down(wide, a)
    mag = f64(wide.abs()) @ f64(a.abs()).T
    assert np.all(np.abs(f64(t) - f64(ref))[:, :r] <= 2.02 * (3 * k + 40) * B.U * mag)


SHAPES = [(1, 1, 256, 1), (1, 8, 256, 16), (2, 40, 512, 7), (16, 264, 256, 8), (17, 257, 768, 13), (63, 512, 1024, 32),
          (64, 1160, 256, 33), (77, 1160, 1280, 8), (130, 520, 512, 64), (300, 72, 2304, 24), (1100, 1032, 256, 16)]


@pytest.mark.parametrize("m,n,k,r", SHAPES)
@pytest.mark.parametrize("ydt,bdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rotate", [False, True])
def test_grad(m, n, k, r, ydt, bdt, rotate):
    d = dev()
    announce("tp_lora_grad_prequantized", m, n, k, r, ydt, bdt, rotate)
    alpha = 0.75
    qa, sa = _codes(m, k, seed=m + k)
    dy, b = _mat((m, n), ydt, seed=n, scale=0.02), _mat((n, r), bdt, seed=n + 1)
    t = torch.zeros((m, 64))
    t[:, :r] = _mat((m, r), F32, seed=n + 2)[:, :r]
    t[:, r:] = 3.0  # not read past the rank
    got = tp.tp_lora_grad_prequantized(_on(d, dy, n), qa.to(d), sa.to(d), t.to(d), _on(d, b, r), alpha, rotate=rotate)
    da, db, dt = (host(v).astype(np.float64) for v in got)
    y64, b64, t64 = f64(dy[:, :n]), f64(b[:, :r]), f64(t[:, :r])
    x = f64(qa) * f64(sa)[:, None]
    wda, wdb, wdt = oracle.lora_grad_codes(y64, qa.numpy(), sa.numpy(), t64, b64, alpha, rotate=rotate)
    mag_dt = alpha * np.abs(y64) @ np.abs(b64)
    terms_dt = n * _parts(ydt, bdt) + 64
    B.assert_sum(dt[:, :r], wdt, mag_dt, terms_dt, "dT")
    assert dt.shape == (m, 64) and np.all(dt[:, r:] == 0)
    B.assert_sum(db, wdb, alpha * np.abs(y64).T @ np.abs(t64), m * _parts(ydt, F32) + 64, "dB")
    # dA is summed from the computed dT: its error, three parts a row, and 8
    # butterfly stages where it is rotated back
    mag_da = mag_dt.T @ np.abs(x)
    if rotate:
        mag_da = B.group_l1(mag_da) / 16.0
    B.assert_sum(da, wda, mag_da, terms_dt + 4 + 3 * m + 64 + (8 if rotate else 0), "dA")


def test_grad_outputs_in_views_and_repeatable():
    d = dev()
    announce("tp_lora_grad_prequantized views, repeats")
    m, n, k, r = 90, 333, 768, 13
    qa, sa = _codes(m, k, seed=9)
    dy, b = _mat((m, n), BF16, seed=10), _mat((n, r), BF16, seed=11)
    t = torch.zeros((m, 64))
    t[:, :r] = _mat((m, r), F32, seed=12)[:, :r]
    args = (_on(d, dy, n), qa.to(d), sa.to(d), t.to(d), _on(d, b, r), 2.0)
    want = tp.tp_lora_grad_prequantized(*args, rotate=True)
    need = tp.tp_lora_grad_workspace_size(m, n, k, r)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=d)
    dab = torch.full((r + 2, k + 8), 7.0, device=d)
    dbb = torch.full((n + 2, r + 3), 7.0, device=d)
    dtb = torch.full((m + 2, 64), 7.0, device=d)
    da, db, dt = tp.tp_lora_grad_prequantized(*args, rotate=True, da=dab[1:-1, 4:4 + k], db=dbb[1:-1, 1:1 + r],
                                              dt=dtb[1:-1], workspace=ws[:need])
    for g, w in zip((da, db, dt), want):
        assert torch.equal(g, w), "the same inputs give the same bytes"
    assert torch.all(dab[0] == 7) and torch.all(dab[-1] == 7) and torch.all(dab[:, :4] == 7)
    assert torch.all(dab[:, 4 + k:] == 7) and torch.all(dbb[0] == 7) and torch.all(dbb[-1] == 7)
    assert torch.all(dbb[:, :1] == 7) and torch.all(dbb[:, 1 + r:] == 7)
    assert torch.all(dtb[0] == 7) and torch.all(dtb[-1] == 7) and torch.all(ws[need:] == 0xA5)


def test_grad_of_nothing():
    d = dev()
    announce("tp_lora_grad_prequantized empty")
    k, r = 512, 5
    b = _mat((24, r), BF16, seed=1)
    da, db, dt = tp.tp_lora_grad_prequantized(
        torch.empty((0, 24), device=d), torch.empty((0, k), dtype=torch.int8, device=d), torch.empty((0,), device=d),
        torch.empty((0, 64), device=d), _on(d, b, r), 1.0)
    assert torch.all(da == 0) and torch.all(db == 0) and db.shape == (24, r) and dt.shape == (0, 64)
    qa, sa = _codes(6, k, seed=2)
    da, db, dt = tp.tp_lora_grad_prequantized(
        torch.empty((6, 0), device=d), qa.to(d), sa.to(d), torch.zeros((6, 64), device=d),
        torch.empty((0, r), dtype=BF16, device=d), 1.0, rotate=True)
    assert torch.all(da == 0) and db.shape == (0, r) and torch.all(dt == 0)
    assert tp.tp_lora_down_prequantized(torch.empty((0, k), dtype=torch.int8, device=d), torch.empty((0,), device=d),
                                        torch.ones((r, k), device=d)).shape == (0, 64)
