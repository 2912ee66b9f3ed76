"""Pins of the oracle's branch operators: published vectors, closed forms,
exhaustive tables and gradients against central differences (fp64, CPU)."""

import numpy as np
import pytest
import torch

import oracle
from tests.test_block_oracle import _differences


def test_philox_known_answers():
    """The generator's published known-answer vectors."""
    for ctr, key, want in [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]:
        assert oracle.philox4x32_10(np.array([ctr], dtype=np.uint64), key)[0].tolist() == list(want)


def test_mask_layout():
    """Element j of run R: 16 bits of word j % 8 // 2, low half first, of the
    counter (R, offset); rows start new runs."""
    seed, offset, m, k, p = 0x123456789ABCDEF0, 0xFEDCBA9876543210, 3, 13, 0.5
    keep = oracle.drop_keep(seed, offset, m, k, p)
    for r in range(m):
        for j in range(k):
            run = r * 2 + j // 8
            w = oracle.philox4x32_10(np.array([[run, 0, offset & 0xFFFFFFFF, offset >> 32]], dtype=np.uint64),
                                     (seed & 0xFFFFFFFF, seed >> 32))[0]
            bits = (int(w[j % 8 // 2]) >> (16 * (j % 2))) & 0xFFFF
            assert keep[r, j] == (bits >= 32768)
    assert np.array_equal(oracle.drop_keep(seed, offset, m, k, p, rows=[2]), keep[2:])
    # runs past 2^32 carry into the counter's second word
    far = oracle.drop_keep(seed, offset, 0, 8, p, rows=[2 ** 32 + 5])
    w = oracle.philox4x32_10(np.array([[5, 1, offset & 0xFFFFFFFF, offset >> 32]], dtype=np.uint64),
                             (seed & 0xFFFFFFFF, seed >> 32))[0]
    assert far[0].tolist() == [((int(w[j // 2]) >> (16 * (j % 2))) & 0xFFFF) >= 32768 for j in range(8)]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.25, 0.5, 0.9, 1.0])
def test_mask_frequency_and_mean(p):
    """2^18 draws: the share that drops within five standard deviations of the
    threshold's, and the factor that keeps the mean."""
    keep = oracle.drop_keep(7, 11, 256, 1024, p)
    q = oracle.drop_threshold(p) / 65536
    assert abs(np.mean(~keep) - q) <= 5 * np.sqrt(q * (1 - q) / keep.size)
    if p < 1:
        assert abs(float(oracle.drop_factor(p)) * (1 - q) - 1) <= 2 ** -24
    x = np.full(keep.shape, 2.0, dtype=np.float32)
    y = oracle.dropout(x, keep, p, None, False)
    assert np.all(y[keep] == (np.float32(2) * oracle.drop_factor(p) if p else 2)) and np.all(y[~keep] == 0)


def test_dropout_gradient_is_the_call_itself():
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((2, 24)), rng.standard_normal((2, 24))
    keep = oracle.drop_keep(1, 2, 2, 24, 0.25)
    f = float(oracle.drop_factor(0.25))
    grad = _differences(lambda v: np.sum(dy * np.where(keep, v * f, 0.0)), x.copy())
    assert np.allclose(oracle.dropout(dy.astype(np.float32), keep, 0.25, None, False), grad, rtol=1e-6, atol=1e-7)


def test_layernorm_closed_forms():
    t = np.full((1, 256), 3.0)
    assert np.all(oracle.layernorm(t, None, None, 1e-5) == 0.0)
    assert np.allclose(oracle.layernorm(t, None, np.arange(256.0), 1e-5), np.arange(256.0))
    t = 5.0 + np.array([[1.0, -1.0] * 128])
    assert np.allclose(oracle.layernorm(t, None, None, 3.0), (t - 5.0) / 2.0, rtol=1e-15)
    rng = np.random.default_rng(5)
    t = rng.standard_normal((4, 512)) + 100.0
    h = oracle.layernorm(t, None, None, 1e-30)
    assert np.allclose(h.mean(axis=1), 0, atol=1e-13) and np.allclose((h * h).mean(axis=1), 1, rtol=1e-12)
    want = torch.nn.functional.layer_norm(torch.from_numpy(t), (512,), eps=1e-5).numpy()
    assert np.allclose(oracle.layernorm(t, None, None, 1e-5), want, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("rotate", [False, True])
def test_layernorm_gradient_against_differences(rotate):
    rng = np.random.default_rng(3)
    t = rng.standard_normal((2, 256)) * 2.0 + 1.0
    gamma, beta = 1.0 + 0.2 * rng.standard_normal(256), 0.1 * rng.standard_normal(256)
    dy, ds = rng.standard_normal((2, 256)), rng.standard_normal((2, 256))

    def loss(t, gamma, beta):
        h = oracle.layernorm(t, gamma, beta, 1e-3)
        return np.sum(dy * (oracle.rotate_groups(h) if rotate else h)) + np.sum(ds * t)

    dx, dgamma, dbeta = oracle.layernorm_backward(dy, t, gamma, 1e-3, dsum=ds, rotate=rotate)
    assert np.allclose(dx, _differences(lambda v: loss(v, gamma, beta), t.copy()), rtol=1e-6, atol=1e-6)
    assert np.allclose(dgamma, _differences(lambda v: loss(t, v, beta), gamma.copy()), rtol=1e-6, atol=1e-6)
    assert np.allclose(dbeta, _differences(lambda v: loss(t, gamma, v), beta.copy()), rtol=1e-6, atol=1e-6)


def test_e4m3_table_is_the_formats():
    """All 256 codes against torch's type, and every code is its own nearest."""
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.e4m3_value(codes)
    assert np.array_equal(got, want, equal_nan=True) and got[0x7E] == 448.0 and got[1] == 2.0 ** -9
    fine = codes[(codes & 0x7F) != 0x7F]
    assert np.array_equal(oracle.e4m3_code(oracle.e4m3_value(fine)), fine)


def test_e4m3_rounding():
    """Midpoints go to the even code, their neighbours to the nearer one; what
    is beyond 448 saturates; subnormals; agreement with torch's conversion."""
    v = oracle.e4m3_value(np.arange(127))
    for i in range(126):
        mid = (v[i] + v[i + 1]) / 2
        even = i if i % 2 == 0 else i + 1
        assert oracle.e4m3_code([mid, np.nextafter(mid, 1e9), np.nextafter(mid, 0)]).tolist() == [even, i + 1, i]
        assert oracle.e4m3_code([-mid])[0] == 0x80 | even
    assert oracle.e4m3_code([449.0, 1e30, -1e30]).tolist() == [0x7E, 0x7E, 0xFE]
    x = np.random.default_rng(1).standard_normal(100000).astype(np.float32) * np.float32(3.0)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_code(x.astype(np.float64)), want)


def test_quantizers():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((130, 200))
    c, s = oracle.quantize_fp8_rows(x)
    assert c.shape == (130, 256) and s.shape == (2, 130) and s.dtype == np.float32
    assert np.all(c[:, 200:] == 0)
    for r in (0, 129):
        for g, (a, b) in enumerate(((0, 128), (128, 200))):
            assert s[g, r] == np.float32(np.abs(x[r, a:b]).max() / 448)
            v = oracle.e4m3_value(c[r, a:b]) * float(s[g, r])
            # half a step: 2^-4 of the value, or of the smallest normal code's
            assert np.all(np.abs(v - x[r, a:b]) <= np.maximum(np.abs(x[r, a:b]), 2.0 ** -6 * s[g, r]) * 2.0 ** -4 * 1.0001)
    ct, st = oracle.quantize_fp8_cols(x)
    c2, s2 = oracle.quantize_fp8_rows(x.T)
    assert np.array_equal(ct, c2) and np.array_equal(st, s2) and ct.shape == (200, 256)
    cb, sb = oracle.quantize_fp8_blocks(x)
    assert cb.shape == (130, 256) and sb.shape == (2, 2)
    assert sb[1, 1] == np.float32(np.abs(x[128:, 128:]).max() / 448)
    tb, stb = oracle.quantize_fp8_blocks(x.T)  # a transposed block is the same block
    assert np.array_equal(tb[:, :130], cb[:, :200].T) and np.array_equal(stb, sb.T)
    z, sz = oracle.quantize_fp8_rows(np.zeros((2, 128)))
    assert not z.any() and not sz.any()


@pytest.mark.parametrize("rows", [1, 128])
def test_product_against_a_loop(rows):
    rng = np.random.default_rng(7)
    a, sa = oracle.quantize_fp8_rows(rng.standard_normal((3, 256)))
    w = rng.standard_normal((130, 256))
    b, sb = oracle.quantize_fp8_rows(w) if rows == 1 else oracle.quantize_fp8_blocks(w)
    c, mag = oracle.qgemm_fp8(a, sa, b, sb, rows)
    for i in range(3):
        for j in (0, 127, 128, 129):
            want = 0.0
            for q in range(256):
                s = sb[q // 128, j] if rows == 1 else sb[j // 128, q // 128]
                want += float(sa[q // 128, i]) * float(s) * oracle.e4m3_value(a[i, q]) * oracle.e4m3_value(b[j, q])
            assert abs(c[i, j] - want) <= 1e-12 * mag[i, j]
