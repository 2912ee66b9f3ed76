"""The precision of fp32 operands of the side path: three bf16 parts, of two such
operands the six products that reach above 2^-24 of the whole.

A dense sum's bound grows with its terms and hides a lost part. Here every
result is ONE product (one code of a row, one gradient of a row or a column),
so it is off by no more than its own roundings, in units of U = 2^-24 of it:

  matrix unit     the parts' products are exact; each step of the sum rounds to
                  fp32 (one unit, two if it truncates), and all but the last are
                  at most 2^-7 of the whole: 2.1
  left-out parts  (1, 2) and (2, 1) of two fp32 operands: a part is at most 2^-8
                  of the one before, so 2 * 2^-24: 2; (2, 2): 2^-32
  factors         sa, alpha: one rounding each: 1

A third part left out is up to 2^-16 of the value, 256 units. The CPU tests plant
that loss (and the other parts') in the oracle's arithmetic and see it caught."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
from tests.gpu_util import announce, dev, f64, host

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
ONE_SPLIT, TWO_SPLITS = 3.2, 5.2  # units, with one factor; another factor adds one


def _check(got, want, units, what):
    off = np.abs(got - want)
    bad = ~(off <= units * U * np.abs(want) + 2.0 ** -140)
    assert not np.any(bad), (f"{what}: {int(bad.sum())} of {bad.size} values out of bounds, worst "
                             f"{float(np.max(off[bad] / (U * np.abs(want[bad]) + 1e-300))):.1f} units")


def _values(shape, dtype, seed):
    """Values over a few binades, away from zero, in rows of 16 bytes."""
    rng = np.random.default_rng(seed)
    v = rng.uniform(1.0, 2.0, size=shape) * 2.0 ** rng.integers(-3, 4, size=shape) * rng.choice([-1.0, 1.0], size=shape)
    pitch = -(-shape[1] // 8) * 8
    full = torch.full((shape[0], pitch), float("nan"), dtype=dtype)
    full[:, :shape[1]] = torch.from_numpy(v.astype(np.float32)).to(dtype)
    return full[:, :shape[1]]


def _on(d, v):
    """On the device with the same (padded) pitch."""
    out = torch.empty((v.shape[0], v.stride(0)), dtype=v.dtype, device=d)[:, :v.shape[1]]
    return out.copy_(v)


def _one_a_row(shape, dtype, seed):
    """One nonzero a row, the columns spread over all of them."""
    m, n = shape
    rng = np.random.default_rng(seed)
    at = (np.arange(m) * 37 + rng.integers(0, n, size=m)) % n
    at[0], at[-1] = 0, n - 1
    v = torch.zeros((m, -(-n // 8) * 8), dtype=dtype)
    v[torch.arange(m), torch.from_numpy(at)] = _values((m, 1), dtype, seed + 1)[:, 0]
    return v[:, :n]


def _one_a_column(shape, dtype, seed):
    m, n = shape
    v = torch.zeros((m, -(-n // 8) * 8), dtype=dtype)
    v[:, :n] = _one_a_row((n, m), dtype, seed)[:, :m].t()
    return v[:, :n]


def _sparse_codes(m, k, seed, by_column):
    rng = np.random.default_rng(seed)
    v = (_one_a_column if by_column else _one_a_row)((m, k), F32, seed)[:, :k].numpy() != 0
    q = rng.integers(1, 128, size=(m, k)) * rng.choice([-1, 1], size=(m, k))
    return torch.from_numpy((v * q).astype(np.int8)), torch.from_numpy(rng.uniform(1e-3, 0.1, size=m).astype(np.float32))


RANKS = [1, 8, 16, 24, 32, 33, 64]


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(1, 256), (16, 2048), (17, 768), (64, 512), (130, 4096)])
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("adt", [BF16, F32])
def test_down_of_one_code_a_row(m, k, r, adt):
    d = dev()
    announce("tp_lora_down_prequantized one code a row", m, k, r, adt)
    qa, sa = _sparse_codes(m, k, m + k, False)
    a = _values((r, k), adt, r)
    t = host(tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), _on(d, a))).astype(np.float64)
    want = (f64(qa) @ f64(a).T) * f64(sa)[:, None]
    _check(t[:, :r], want, ONE_SPLIT, "T")


SHAPES = [(1, 8, 256), (16, 264, 512), (17, 1160, 256), (64, 520, 512), (130, 257, 768)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("ydt,bdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_gradients_of_one_product_each(m, n, k, r, ydt, bdt):
    d = dev()
    announce("tp_lora_grad_prequantized one product", m, n, k, r, ydt, bdt)
    alpha = 0.7
    a32 = float(np.float32(alpha))
    qa, sa = _sparse_codes(m, k, k + m, True)
    b, t = _values((n, r), bdt, n), torch.zeros((m, 64))
    t[:, :r] = _values((m, r), F32, n + 1)
    both = TWO_SPLITS if ydt == F32 and bdt == F32 else ONE_SPLIT
    # one gradient a row: dT; one code a column: dA, from the dT that came out
    dy = _one_a_row((m, n), ydt, m)
    da, _, dt = tp.tp_lora_grad_prequantized(_on(d, dy), qa.to(d), sa.to(d), t.to(d), _on(d, b), alpha)
    dt64 = f64(dt)[:, :r]
    _check(dt64, a32 * (f64(dy) @ f64(b)), both, "dT")
    _check(f64(da), (dt64 * f64(sa)[:, None]).T @ f64(qa), ONE_SPLIT, "dA")
    # one gradient a column: dB
    dy = _one_a_column((m, n), ydt, m + 1)
    _, db, _ = tp.tp_lora_grad_prequantized(_on(d, dy), qa.to(d), sa.to(d), t.to(d), _on(d, b), alpha)
    _check(f64(db), a32 * (f64(dy).T @ f64(t)[:, :r]), TWO_SPLITS if ydt == F32 else ONE_SPLIT, "dB")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 40, 130])
@pytest.mark.parametrize("r", [8, 64])
def test_down_at_the_ends_of_an_fp32_operand(m, r):
    """Values of 2^-100, whose third part is still a normal number, count in full;
    one that bf16 rounds to infinity makes its own rank NaN and no other."""
    d = dev()
    announce("tp_lora_down_prequantized ends of fp32", m, r)
    k = 512
    qa, _ = _sparse_codes(m, k, m, False)
    sa = torch.ones(m)
    a = _values((r, k), F32, r)
    small = (a * 2.0 ** -100).contiguous()
    t = tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), small.to(d))
    _check(f64(t)[:, :r], f64(qa) @ f64(small).T, ONE_SPLIT, "T")
    whole = tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), a.contiguous().to(d))
    large = a.contiguous()
    large[r // 2, 3] = 3.4e38
    t = tp.tp_lora_down_prequantized(qa.to(d), sa.to(d), large.to(d))
    keep = [j for j in range(64) if j != r // 2]
    assert torch.all(torch.isnan(t[:, r // 2])) and torch.equal(t[:, keep], whole[:, keep])


# ----------------------------------------------------------- planted on the CPU
def _bf16(v):
    return torch.from_numpy(v.astype(np.float32)).to(BF16).double().numpy()


def _parts(v):
    hi = _bf16(v)
    mid = _bf16(v - hi)
    return hi, mid, _bf16(v - hi - mid)


def _products(x, y, keep):
    xs, ys = _parts(x), _parts(y)
    return sum(xs[i] * ys[j] for i in range(3) for j in range(3) if keep(i, j))


def _operands():
    x = f64(_values((40, 24), F32, 5))
    return x, f64(_values((40, 24), F32, 6))


def test_six_products_are_inside_the_bound():
    x, y = _operands()
    assert all(np.array_equal(sum(_parts(v)), v) for v in (x, y))
    _check(_products(x, y, lambda i, j: i + j <= 2), x * y, TWO_SPLITS - 3.1, "six products")


@pytest.mark.parametrize("lost", [(0, 1), (1, 0), (0, 2), (1, 1), (2, 0)])
def test_a_lost_product_is_caught(lost):
    x, y = _operands()
    with pytest.raises(AssertionError):
        _check(_products(x, y, lambda i, j: i + j <= 2 and (i, j) != lost), x * y, TWO_SPLITS, "product")


@pytest.mark.parametrize("parts", [1, 2])
def test_a_lost_part_of_one_operand_is_caught(parts):
    x, _ = _operands()
    codes = np.random.default_rng(1).integers(1, 128, size=x.shape)
    with pytest.raises(AssertionError):
        _check(sum(_parts(x)[:parts]) * codes, x * codes, ONE_SPLIT, "product")
