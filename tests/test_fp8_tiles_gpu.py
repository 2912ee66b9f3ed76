"""The main loops of tp_qgemm_fp8's tiles over many blocks of k: every stage of
their rings filled again and again, odd and even numbers of steps, both layouts
of b's scales with another scale in every block. Exactly, on whole numbers; and
the 8-bit matrix instruction's sums by what is left of them where the products
cancel."""

import numpy as np
import pytest
import torch

import int4_quantized_gemm_amd as tp
import oracle
from tests.fp8_plan import LOST_8BIT, plan
from tests.gpu_util import announce, dev, f64

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn

# m, n, blocks of k, type, the tile it is meant to reach and its splits
LOOPS = [
    (1999, 4093, (5, 8, 9), BF16, (128, 128), 1),
    (1999, 4093, (5, 8, 9), F32, (128, 128), 1),
    (4093, 4091, (6,), F32, (128, 128), 1),
    (4093, 4091, (5, 8, 9), BF16, (256, 256), 1),
    (300, 4096, (3, 4, 5, 10, 17), BF16, (64, 128), 1),
    (300, 4096, (3, 4, 5, 10, 17), F32, (64, 128), 1),
]


def _whole(r, k, g, d):
    return torch.randint(-8, 9, (r, k), generator=g, device=d).float()


@pytest.mark.parametrize("m,n,blocks,dtype,tile,splits", LOOPS)
@pytest.mark.parametrize("rows", [128, 1])
def test_many_steps_exact(m, n, blocks, dtype, tile, splits, rows):
    d = dev()
    for kb in blocks:
        k = 128 * kb
        assert plan(m, n, k, dtype == BF16) == (tile, splits)
        announce("tp_qgemm_fp8 many steps", m, n, k, rows, dtype)
        g = torch.Generator(device=d).manual_seed(m + n + k + rows)
        a, b = _whole(m, k, g, d), _whole(n, k, g, d)
        pow2 = lambda *s: 2.0 ** torch.randint(-2, 2, s, generator=g, device=d).float()  # noqa: E731
        sa = pow2(kb, m)
        sb = pow2(kb, n) if rows == 1 else pow2(-(-n // 128), kb)
        full = sb.t().repeat_interleave(128, 1) if rows == 1 else sb.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        assert 64 * k * 4 * 16 < 2 ** 24  # multiples of 1/16 below 2^20: exact in any order
        want = (a * sa.t().repeat_interleave(128, 1)).double() @ (b * full).double().t().contiguous()
        # a few rows on the host, from the oracle
        for i in (0, m // 2, m - 1):
            c, _ = oracle.qgemm_fp8(oracle.e4m3_code(f64(a[i:i + 1])), f64(sa[:, i:i + 1]), oracle.e4m3_code(f64(b)), f64(sb), rows)
            assert np.array_equal(want[i].cpu().numpy(), c[0])
        args = (a.to(F8), sa, b.to(F8), sb)
        got = tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=dtype)
        assert torch.equal(got, want.to(dtype)), f"k={k}: {int((got != want.to(dtype)).sum())} values differ"
        for _ in range(3):  # a load that came too late would not come too late every time
            assert torch.equal(tp.tp_qgemm_fp8(*args, b_block_rows=rows, out_dtype=dtype), got)


def _halves(m, n, g, d, loud):
    """Codes [m, 256], [n, 256] whose second block is the first one in another order
    and with the other sign: their product is 0, and what comes out is the
    difference of two blocks' sums as the matrix instruction takes them."""
    x = torch.randn((m, 128), generator=g, device=d)
    if loud:  # one channel 100 times the others
        x[:, 77] *= 100.0
    a, _ = tp.tp_quantize_fp8(x)
    b, _ = tp.tp_quantize_fp8(torch.randn((n, 128), generator=g, device=d))
    order = torch.randperm(128, generator=g, device=d)
    turn = lambda q, sign: torch.cat([q.float(), sign * q.float()[:, order]], 1).to(F8)  # noqa: E731
    return turn(a, 1.0), turn(b, -1.0), a.float(), b.float()


@pytest.mark.parametrize("m,n,dtype", [(300, 4096, BF16), (1999, 4093, BF16), (4093, 4091, BF16), (300, 4096, F32), (1999, 4093, F32), (12, 4096, BF16)])
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("loud", [False, True])
def test_what_a_block_s_sum_loses(m, n, dtype, rows, loud):
    """Where C is bf16, on tiles, the 8-bit instruction loses at most LOST_8BIT of the
    sums' norm, so the difference of two sums at most twice that. (bf16's rounding is
    that of the small difference: it does not hide it.) Elsewhere the sums are fp32's:
    each of at most 128 additions rounds by at most 2^-23 of a running sum whose norm
    is not above the whole's; the roundings of different additions have independent
    signs, so 128^(1/2) 2^-23 of the norm, and 2^(1/2) times that for the difference."""
    d = dev()
    announce("what a block's sum loses", m, n, dtype, rows, loud)
    g = torch.Generator(device=d).manual_seed(m + n + loud)
    a, b, ah, bh = _halves(m, n, g, d, loud)
    one = lambda *s: torch.ones(s, device=d)  # noqa: E731
    c = tp.tp_qgemm_fp8(a, one(2, m), b, one(2, n) if rows == 1 else one(-(-n // 128), 2), b_block_rows=rows, out_dtype=dtype)
    size = (ah.double() @ bh.double().t().contiguous()).norm()
    lost = float(c.double().norm() / size)
    print("lost", lost, flush=True)
    eight_bit = dtype == BF16 and plan(m, n, 256, True)[0] != "few"
    assert lost <= (2 * LOST_8BIT if eight_bit else 256 ** 0.5 * 2.0 ** -23)


@pytest.mark.parametrize("m,n,k", [(300, 4096, 640), (1999, 4093, 640), (1999, 4093, 1152), (4093, 4091, 640), (4093, 4091, 1152)])
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("loud", [False, True])
def test_quantized_data_in_the_norm(m, n, k, rows, loud):
    """bf16 C against the exact result rounded once. An output that is off by e before
    its rounding rounds the other way with a chance of |e| over the distance u of its
    two neighbours, and is then off by u: the square of the difference's norm is
    sum |e| u in the mean, at most ||e|| ||u|| <= LOST_8BIT 2^-7 of the norm's square."""
    d = dev()
    announce("tp_qgemm_fp8 in the norm", m, n, k, rows, loud)
    g = torch.Generator(device=d).manual_seed(m + n + k)
    x = torch.randn((m, k), generator=g, device=d)
    if loud:
        x[:, ::200] *= 30.0
    a, sa = tp.tp_quantize_fp8(x)
    b, sb = tp.tp_quantize_fp8(torch.randn((n, k), generator=g, device=d), block_rows=rows)
    full = sb.t().repeat_interleave(128, 1) if rows == 1 else sb.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    exact = (a.double() * sa.double().t().repeat_interleave(128, 1)) @ (b.double() * full.double()).t().contiguous()
    got = tp.tp_qgemm_fp8(a, sa, b, sb, b_block_rows=rows, out_dtype=BF16)
    off = float((got.double() - exact.to(BF16).double()).norm() / exact.norm())
    print("off", off, flush=True)
    assert off <= (LOST_8BIT * 2.0 ** -7) ** 0.5
