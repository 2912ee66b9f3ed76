"""Refusals of dropout, layer norm and the 8-bit float products, without a GPU:
every invalid call is named before any HIP call (made-up device addresses;
nothing is dereferenced or launched), and the binding refuses what the C
boundary cannot see."""

import os

import pytest
import torch

import int4_quantized_gemm_amd as tp
from int4_quantized_gemm_amd import _lib

# disjoint fake addresses
A, B, C, D, E, F, G, H, I, J, K = (0x100000000 * i for i in range(1, 12))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _lib.load()


def _err(lib):
    return lib.tp_last_error_message().decode()


# ------------------------------------------------------------------- dropout
def dr(lib, x=A, xdt=0, ldx=100, res=B, ldr=100, p=0.1, rng=C, m=7, k=99, y=D, ydt=0, ldy=100):
    return lib.tp_dropout(x, xdt, ldx, res, ldr, p, rng, m, k, y, ydt, ldy, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 2), (dict(k=-1), 2), (dict(m=2 ** 31), 2), (dict(k=2 ** 31, ldx=2 ** 31, ldr=2 ** 31, ldy=2 ** 31), 2),
    (dict(x=0), 1), (dict(y=0), 1), (dict(rng=0), 1),
    (dict(ldx=96), 4), (dict(ldr=96), 4), (dict(ldy=0), 4), (dict(ldx=-4), 4),
    (dict(x=A + 8), 5), (dict(res=B + 4), 5), (dict(y=D + 8), 5), (dict(ldx=99), 5), (dict(ldy=101), 5), (dict(rng=C + 4), 5),
    (dict(xdt=2), 6), (dict(ydt=-1), 6), (dict(ldx=2 ** 62), 8),
    (dict(p=-0.1), 13), (dict(p=1.0001), 13), (dict(p=float("nan")), 13), (dict(p=float("inf")), 13),
    (dict(y=A + 400), 10), (dict(y=B + 1600), 10), (dict(y=C - 400), 10), (dict(y=A, ydt=1, ldr=104, ldy=200), 10), (dict(y=A, ldy=104), 10),
])
def test_dropout_refusals(lib, kw, status):
    assert dr(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_dropout_empty(lib):
    assert dr(lib, m=0) == 0 and dr(lib, k=0) == 0
    assert dr(lib, m=0, x=0, res=0, y=0) == 0
    assert dr(lib, m=0, p=0.0, rng=0) == 0      # nothing drops: no generator


# ---------------------------------------------------------------- layer norm
def ln(lib, x=A, xdt=0, ldx=512, res=B, ldr=512, sm=C, lds=512, sdt=0, g=D, b=E, gdt=0, eps=1e-5, p=0.1, rng=F, fl=1,
       m=64, k=512, kind=2, y=G, ldy=512, sc=H, ldsc=64):
    return lib.tp_layernorm_rotate(x, xdt, ldx, res, ldr, sm, lds, sdt, g, b, gdt, eps, p, rng, fl, m, k, kind, y, ldy,
                                   sc, ldsc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=0), 2), (dict(m=-1), 2), (dict(m=2 ** 31), 2),
    (dict(k=16640, ldx=16640, ldr=16640, lds=16640, ldy=16640), 2),
    (dict(x=0), 1), (dict(y=0), 1), (dict(sc=0), 1), (dict(kind=0, sc=0), 1), (dict(res=0), 1), (dict(sm=0), 1), (dict(rng=0), 1),
    (dict(res=0, sm=0), 1),                     # a dropout without a residual
    (dict(ldx=500), 4), (dict(ldr=511), 4), (dict(lds=0), 4), (dict(ldy=511), 4), (dict(kind=1, ldy=500), 4), (dict(ldsc=63), 4),
    (dict(x=A + 8), 5), (dict(res=B + 4), 5), (dict(sm=C + 8), 5), (dict(g=D + 8), 5), (dict(b=E + 4), 5), (dict(y=G + 1), 5),
    (dict(sc=H + 2), 5), (dict(ldx=513), 5), (dict(rng=F + 4), 5),
    (dict(xdt=2), 6), (dict(sdt=5), 6), (dict(gdt=-1), 6), (dict(g=0, gdt=3), 6),
    (dict(kind=3), 11), (dict(kind=-1), 11), (dict(fl=2), 11),
    (dict(eps=0.0), 13), (dict(eps=float("nan")), 13), (dict(eps=9e-31), 13), (dict(eps=1.1e30), 13),
    (dict(p=-1e-9), 13), (dict(p=1.5), 13), (dict(p=float("nan")), 13),
    (dict(ldx=2 ** 62), 8),
    (dict(y=A + 4096), 10), (dict(y=B), 10), (dict(y=C), 10), (dict(y=D), 10), (dict(y=E), 10), (dict(y=F), 10), (dict(sc=G + 64), 10),
    (dict(sc=A), 10), (dict(sc=F), 10), (dict(sm=D), 10), (dict(sm=E), 10), (dict(sm=F - 512), 10), (dict(sm=B + 16), 10),
    (dict(sm=B, lds=516), 10), (dict(sm=A, sdt=1), 10), (dict(sm=A + 2048), 10),
])
def test_layernorm_refusals(lib, kw, status):
    assert ln(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_layernorm_empty_and_optional(lib):
    assert ln(lib, m=0) == 0
    assert ln(lib, m=0, x=0, res=B, y=0, sc=0) == 0
    assert ln(lib, m=0, x=0, res=0, sm=0, y=0, sc=0) == 0  # with a dropout
    assert ln(lib, m=0, res=0, sm=0, g=0, b=0, gdt=9, sdt=9, p=0.0, rng=0) == 0
    assert ln(lib, m=0, kind=1, sc=0, ldsc=0) == 0
    assert ln(lib, m=0, kind=0, ldsc=0) == 0


def lb(lib, dy=A, ydt=0, lddy=512, fl=1, t=B, tdt=0, ldt=512, g=C, gdt=0, eps=1e-5, ds=D, ldds=512, p=0.1, rng=E, m=64, k=512,
       dx=F, xdt=0, lddx=512, br=G, lddb=512, dg=H, db=I, ws=J, wsb=1 << 24):
    return lib.tp_layernorm_rotate_backward(dy, ydt, lddy, fl, t, tdt, ldt, g, gdt, eps, ds, ldds, p, rng, m, k, dx, xdt, lddx,
                                            br, lddb, dg, db, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=-256), 2), (dict(m=-1), 2), (dict(k=16640), 2),
    (dict(dy=0), 1), (dict(t=0), 1), (dict(dx=0), 1), (dict(rng=0), 1),
    (dict(lddy=500), 4), (dict(ldt=500), 4), (dict(ldds=500), 4), (dict(lddx=500), 4), (dict(lddb=500), 4),
    (dict(dy=A + 8), 5), (dict(t=B + 2), 5), (dict(g=C + 4), 5), (dict(ds=D + 8), 5), (dict(dx=F + 8), 5), (dict(br=G + 8), 5),
    (dict(dg=H + 1), 5), (dict(db=I + 2), 5), (dict(ws=J + 8), 5), (dict(rng=E + 2), 5),
    (dict(ydt=2), 6), (dict(tdt=2), 6), (dict(xdt=2), 6), (dict(gdt=2), 6),
    (dict(fl=3), 11), (dict(eps=0.0), 13), (dict(p=2.0), 13), (dict(ldt=2 ** 62), 8),
    (dict(ws=0), 9), (dict(wsb=100), 9), (dict(ws=0, dg=0), 9),
    (dict(dx=A), 10), (dict(dx=A, dg=0), 10), (dict(dx=A, db=0), 10), (dict(dx=B), 10), (dict(dx=C), 10), (dict(dx=E), 10), (dict(dx=A, ydt=1), 10), (dict(dx=A + 16), 10), (dict(dx=D, lddx=516), 10),
    (dict(br=A), 10), (dict(br=B), 10), (dict(br=D), 10), (dict(br=F), 10), (dict(br=H), 10), (dict(br=I), 10), (dict(br=E), 10),
    (dict(dg=F), 10), (dict(dg=A), 10), (dict(db=H + 4), 10), (dict(ws=A), 10), (dict(ws=F), 10), (dict(ws=H), 10), (dict(ws=G), 10),
])
def test_layernorm_backward_refusals(lib, kw, status):
    assert lb(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_layernorm_backward_empty_and_workspace(lib):
    assert lb(lib, m=0, dg=0, db=0, ws=0) == 0
    for k in (256, 4096, 4352, 16384):
        assert lib.tp_layernorm_backward_workspace_size(64, k) >= 2 * k * 4
    for m, k in ((0, 512), (-1, 512), (4, 300), (4, 0), (4, 16640), (2 ** 31, 256)):
        assert lib.tp_layernorm_backward_workspace_size(m, k) == 0


# ----------------------------------------------------------------- quantizers
def qt(lib, x=A, xdt=0, ldx=512, m=200, k=500, fl=0, br=1, q=B, ldq=512, s=C, lds=200, t=D, ldt=256, st=E, ldst=500):
    return lib.tp_quantize_fp8(x, xdt, ldx, m, k, fl, br, q, ldq, s, lds, t, ldt, st, ldst, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 2), (dict(k=-1), 2), (dict(m=2 ** 26), 2), (dict(k=2 ** 26), 2), (dict(m=2 ** 20, k=2 ** 15), 2),
    (dict(fl=1), 3), (dict(fl=1, k=384), 3),
    (dict(x=0), 1), (dict(q=0), 1), (dict(s=0), 1), (dict(t=0), 1), (dict(st=0), 1), (dict(q=0, s=0, t=0, st=0), 1),
    (dict(ldx=496), 4), (dict(ldq=511), 4), (dict(lds=199), 4), (dict(ldt=255), 4), (dict(ldst=499), 4),
    (dict(br=128, lds=3), 4), (dict(br=128, ldst=1), 4),
    (dict(x=A + 4), 5), (dict(q=B + 8), 5), (dict(ldq=520), 5), (dict(t=D + 1), 5), (dict(s=C + 2), 5), (dict(st=E + 1), 5),
    (dict(xdt=2), 6), (dict(ldx=2 ** 62), 8), (dict(fl=2), 11), (dict(br=2), 11), (dict(br=0), 11),
    (dict(q=A), 10), (dict(s=A + 64), 10), (dict(t=A + 1024), 10), (dict(st=A), 10), (dict(s=B), 10), (dict(t=B), 10), (dict(st=C), 10),
    (dict(st=D + 16), 10),
])
def test_quantizer_refusals(lib, kw, status):
    assert qt(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_quantizer_empty(lib):
    assert qt(lib, m=0) == 0 and qt(lib, k=0) == 0
    assert qt(lib, m=0, x=0, q=0, s=0, t=0, st=0) == 0


# -------------------------------------------------------------------- product
def gm(lib, a=A, lda=512, sa=B, ldsa=300, b=C, ldb=512, sb=D, ldsb=4, br=128, m=300, n=700, k=512, c=E, cdt=0, ldc=700, ws=F,
       wsb=1 << 28):
    return lib.tp_qgemm_fp8(a, lda, sa, ldsa, b, ldb, sb, ldsb, br, m, n, k, c, cdt, ldc, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 2), (dict(n=-1), 2), (dict(k=0), 2), (dict(k=100), 2), (dict(k=-128), 2), (dict(k=2 ** 24), 2), (dict(m=2 ** 26), 2),
    (dict(n=2 ** 26), 2), (dict(m=2 ** 20, n=2 ** 17), 2),
    (dict(a=0), 1), (dict(sa=0), 1), (dict(b=0), 1), (dict(sb=0), 1), (dict(c=0), 1),
    (dict(lda=511), 4), (dict(ldb=496), 4), (dict(ldsa=299), 4), (dict(ldsb=3), 4), (dict(br=1, ldsb=699), 4), (dict(ldc=699), 4),
    (dict(lda=2 ** 24), 4), (dict(ldb=2 ** 24), 4),
    (dict(a=A + 8), 5), (dict(b=C + 4), 5), (dict(lda=520), 5), (dict(sa=B + 1), 5), (dict(sb=D + 2), 5), (dict(c=E + 2), 5),
    (dict(cdt=1, c=E + 1), 5),
    (dict(cdt=2), 6), (dict(br=64), 11), (dict(ldc=2 ** 62), 8), (dict(lda=2 ** 63 - 1), 8),
    (dict(ws=0, m=100, n=100, k=8192, lda=8192, ldb=8192, ldsb=64), 9),
    (dict(wsb=16, m=100, n=100, k=8192, lda=8192, ldb=8192, ldsb=64), 9),
    (dict(ws=F + 8, m=100, n=100, k=8192, lda=8192, ldb=8192, ldsb=64), 5),
    (dict(ws=A, m=100, n=100, k=8192, lda=8192, ldb=8192, ldsb=64), 10),
    (dict(ws=E, m=100, n=100, k=8192, lda=8192, ldb=8192, ldsb=64), 10),
    (dict(c=A), 10), (dict(c=B), 10), (dict(c=C + 1024), 10), (dict(c=D), 10),
])
def test_product_refusals(lib, kw, status):
    assert gm(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_product_empty_and_workspace(lib):
    assert gm(lib, m=0) == 0 and gm(lib, n=0) == 0
    assert gm(lib, m=0, n=0, a=0, sa=0, b=0, sb=0, c=0, ws=0) == 0
    size = lib.tp_qgemm_fp8_workspace_size
    for bf16 in (0, 1):
        assert size(100, 100, 8192, bf16) > 0      # one tile: k is split
        assert size(1, 4096, 12288, bf16) == 0 and size(4096, 12288, 4096, bf16) == 0
        for m, n, k in ((0, 4, 128), (4, 0, 128), (4, 4, 100), (4, 4, 0), (-1, 4, 128), (2 ** 26, 4, 128), (4, 4, 2 ** 24)):
            assert size(m, n, k, bf16) == 0
    assert size(100, 100, 8192, 7) == 0


def test_sizes_at_the_limits_do_not_overflow(lib):
    """The largest sizes that pass the size checks: every extent and workspace
    is computed without overflow (the calls end at a missing pointer)."""
    big = 2 ** 26 - 1
    assert qt(lib, m=big, k=256, ldx=256, ldq=256, lds=big, ldt=2 ** 26, ldst=256, t=0, st=0, q=0) == 1
    assert gm(lib, m=big, n=1, k=128, lda=128, ldb=128, ldsa=big, ldsb=1, ldc=4, c=0) == 1
    assert lib.tp_qgemm_fp8_workspace_size(2 ** 18, 2 ** 18, 2 ** 24 - 128, 0) == 0
    assert lib.tp_layernorm_backward_workspace_size(2 ** 31 - 1, 16384) > (2 ** 31 - 1) * 16


# -------------------------------------------------------------------- binding
def test_binding_refuses_host_tensors():
    x, q = torch.zeros((4, 256)), torch.zeros((4, 256), dtype=torch.float8_e4m3fn)
    s = torch.zeros((2, 4))
    for call in (lambda: tp.tp_dropout(x, 0.1, torch.zeros(2, dtype=torch.int64)), lambda: tp.tp_layernorm_rotate(x),
                 lambda: tp.tp_layernorm_rotate_backward(x, x), lambda: tp.tp_quantize_fp8(x),
                 lambda: tp.tp_qgemm_fp8(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
