"""Refusals of the operators around the projections, without a GPU: every
invalid call is named before any HIP call (made-up device addresses; nothing is
dereferenced or launched), and the binding refuses what the C boundary cannot
see."""

import os

import pytest
import torch

import int4_quantized_gemm_amd as tp
from int4_quantized_gemm_amd import _lib

A, B, C, D, E, F, G = (0x10000000 * i for i in range(1, 8))  # disjoint fake addresses


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _lib.load()


def _err(lib):
    return lib.tp_last_error_message().decode()


# ----------------------------------------------------------------- RMS norm
def nr(lib, x=A, xdt=0, ldx=512, res=B, ldr=512, sm=C, lds=512, sdt=0, g=D, gdt=0, eps=1e-6, fl=1, m=64, k=512,
       kind=0, y=E, ldy=512, sc=F):
    return lib.tp_rmsnorm_rotate(x, xdt, ldx, res, ldr, sm, lds, sdt, g, gdt, eps, fl, m, k, kind, y, ldy, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=0), 2), (dict(m=-1), 2), (dict(m=2 ** 31), 2),
    (dict(k=16640, ldx=16640, ldr=16640, lds=16640, ldy=16640), 2),
    (dict(x=0), 1), (dict(y=0), 1), (dict(sc=0), 1), (dict(res=0), 1), (dict(sm=0), 1),
    (dict(ldx=500), 4), (dict(ldr=511), 4), (dict(lds=0), 4), (dict(ldy=511), 4), (dict(kind=1, ldy=500), 4),
    (dict(x=A + 8), 5), (dict(res=B + 4), 5), (dict(sm=C + 8), 5), (dict(g=D + 8), 5), (dict(y=E + 1), 5),
    (dict(sc=F + 2), 5), (dict(ldx=513), 5),
    (dict(xdt=2), 6), (dict(sdt=5), 6), (dict(gdt=-1), 6),
    (dict(kind=2), 11), (dict(fl=2), 11),
    (dict(eps=0.0), 13), (dict(eps=-1e-6), 13), (dict(eps=float("nan")), 13), (dict(eps=float("inf")), 13),
    (dict(eps=9e-31), 13), (dict(eps=1.1e30), 13),
    (dict(ldx=2 ** 62), 8),
    (dict(y=A + 4096), 10), (dict(y=B), 10), (dict(y=C), 10), (dict(y=D), 10), (dict(sc=E + 64), 10),
    (dict(sc=A), 10), (dict(sm=D), 10), (dict(sm=B + 16), 10), (dict(sm=B, lds=516), 10), (dict(sm=A, sdt=1), 10),
    (dict(sm=A + 2048), 10),
])
def test_norm_refusals(lib, kw, status):
    assert nr(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_norm_empty_and_optional(lib):
    assert nr(lib, m=0) == 0
    assert nr(lib, m=0, x=0, y=0, sc=0) == 0
    assert nr(lib, m=0, res=0, sm=0, g=0, sdt=9) == 0       # no residual, no weight
    assert nr(lib, m=0, kind=1, sc=0) == 0


def nb(lib, dy=A, ydt=0, lddy=512, fl=1, t=B, tdt=0, ldt=512, g=C, gdt=0, eps=1e-6, ds=D, ldds=512, m=64, k=512,
       dx=E, xdt=0, lddx=512, dg=F, ws=G, wsb=1 << 24):
    return lib.tp_rmsnorm_rotate_backward(dy, ydt, lddy, fl, t, tdt, ldt, g, gdt, eps, ds, ldds, m, k, dx, xdt, lddx,
                                          dg, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=-256), 2), (dict(m=-1), 2), (dict(k=16640), 2),
    (dict(dy=0), 1), (dict(t=0), 1), (dict(dx=0), 1),
    (dict(lddy=500), 4), (dict(ldt=500), 4), (dict(ldds=500), 4), (dict(lddx=500), 4),
    (dict(dy=A + 8), 5), (dict(t=B + 2), 5), (dict(g=C + 4), 5), (dict(ds=D + 8), 5), (dict(dx=E + 8), 5),
    (dict(dg=F + 1), 5), (dict(ws=G + 8), 5),
    (dict(ydt=2), 6), (dict(tdt=2), 6), (dict(xdt=2), 6), (dict(gdt=2), 6),
    (dict(fl=3), 11), (dict(eps=0.0), 13), (dict(eps=1e-300), 13), (dict(ldt=2 ** 62), 8),
    (dict(ws=0), 9), (dict(wsb=100), 9),
    (dict(dx=B), 10), (dict(dx=C), 10), (dict(dx=A, ydt=1), 10), (dict(dx=A + 16), 10), (dict(dx=D, lddx=516), 10),
    (dict(dg=E), 10), (dict(dg=A), 10), (dict(ws=A), 10), (dict(ws=E), 10), (dict(ws=F), 10),
])
def test_norm_backward_refusals(lib, kw, status):
    assert nb(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_norm_backward_empty_and_workspace(lib):
    assert nb(lib, m=0, dg=0, ws=0) == 0
    assert lib.tp_rmsnorm_backward_workspace_size(64, 512) > 0
    for m, k in ((0, 512), (-1, 512), (4, 300), (4, 0), (4, 16640), (2 ** 31, 256)):
        assert lib.tp_rmsnorm_backward_workspace_size(m, k) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 256))
    for call in (lambda: tp.tp_rmsnorm_rotate(x), lambda: tp.tp_rmsnorm_rotate_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------- side path on 8-bit activations
def dn(lib, q=A, ldq=512, s=B, a=C, adt=0, lda=512, m=64, k=512, r=16, t=D, tb=1 << 20, ws=E, wsb=1 << 24):
    return lib.tp_lora_down_prequantized(q, ldq, s, a, adt, lda, m, k, r, t, tb, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=0), 2), (dict(m=-1), 2), (dict(r=0), 2), (dict(r=65), 2),
    (dict(q=0), 1), (dict(s=0), 1), (dict(a=0), 1), (dict(t=0), 1),
    (dict(ldq=511), 4), (dict(lda=500), 4), (dict(q=A + 8), 5), (dict(ldq=520), 5), (dict(a=C + 8), 5),
    (dict(s=B + 1), 5), (dict(t=D + 4), 5), (dict(adt=4), 6), (dict(tb=64 * 256 - 1), 9),
    (dict(lda=2 ** 62), 8), (dict(t=A + 1024), 10), (dict(t=B), 10), (dict(t=C), 10), (dict(m=2 ** 27), 2), (dict(m=2 ** 26), 2),
    (dict(ws=0), 9), (dict(wsb=16), 9), (dict(ws=E + 8), 5), (dict(ws=A), 10), (dict(ws=B), 10), (dict(ws=C), 10),
    (dict(ws=D), 10),
])
def test_down_refusals(lib, kw, status):
    assert dn(lib, **kw) == status, _err(lib)
    assert _err(lib)


H, I, J = (0x10000000 * i for i in range(8, 11))


def gr(lib, dy=A, ydt=0, lddy=512, q=B, ldq=512, s=C, t=D, b=E, bdt=0, ldb=16, alpha=1.0, fl=0, m=64, n=512, k=512,
       r=16, dt=F, da=G, ldda=512, db=H, lddb=16, ws=I, wsb=1 << 26):
    return lib.tp_lora_grad_prequantized(dy, ydt, lddy, q, ldq, s, t, b, bdt, ldb, alpha, fl, m, n, k, r, dt, da, ldda,
                                         db, lddb, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=300), 3), (dict(k=0), 2), (dict(m=-1), 2), (dict(n=-1), 2), (dict(r=0), 2), (dict(r=65, ldb=68), 2),
    (dict(m=2 ** 27), 2), (dict(n=2 ** 27, lddy=2 ** 27), 2),
    (dict(m=2 ** 26), 2), (dict(n=2 ** 26, lddy=2 ** 26), 2), (dict(k=2 ** 26, ldq=2 ** 26, ldda=2 ** 26), 2),
    (dict(dy=0), 1), (dict(q=0), 1), (dict(s=0), 1), (dict(t=0), 1), (dict(b=0), 1), (dict(dt=0), 1),
    (dict(da=0), 1), (dict(db=0), 1),
    (dict(lddy=511), 4), (dict(ldq=500), 4), (dict(ldb=15), 4), (dict(ldda=511), 4), (dict(lddb=15), 4),
    (dict(dy=A + 8), 5), (dict(q=B + 4), 5), (dict(b=E + 4), 5), (dict(dt=F + 4), 5), (dict(da=G + 4), 5),
    (dict(db=H + 2), 5), (dict(ws=I + 8), 5), (dict(ldb=17), 5), (dict(ldda=513), 5),
    (dict(ydt=2), 6), (dict(bdt=2), 6), (dict(fl=2), 11), (dict(ws=0), 9), (dict(wsb=16), 9),
    (dict(lddy=2 ** 62), 8),
    (dict(dt=A), 10), (dict(da=B), 10), (dict(db=C), 10), (dict(ws=D), 10), (dict(ws=E), 10), (dict(dt=D), 10),
    (dict(da=F), 10), (dict(db=G), 10), (dict(ws=F), 10), (dict(ws=G), 10), (dict(ws=H), 10),
])
def test_grad_refusals(lib, kw, status):
    assert gr(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_down_workspace_query(lib):
    assert lib.tp_lora_down_prequantized_workspace_size(64, 512, 16) > 0
    for args in ((-1, 256, 4), (0, 256, 4), (8, 300, 4), (8, 0, 4), (8, 256, 0), (8, 256, 65), (2 ** 27, 256, 4), (2 ** 26, 256, 4)):
        assert lib.tp_lora_down_prequantized_workspace_size(*args) == 0


def test_grad_workspace_query(lib):
    assert lib.tp_lora_grad_workspace_size(64, 512, 512, 16) > 0
    for args in ((-1, 8, 256, 4), (8, -1, 256, 4), (8, 8, 300, 4), (8, 8, 0, 4), (8, 8, 256, 0), (8, 8, 256, 65),
                 (2 ** 27, 8, 256, 4), (8, 2 ** 27, 256, 4), (2 ** 26, 8, 256, 4), (8, 2 ** 26, 256, 4),
                 (8, 8, 2 ** 26, 4)):
        assert lib.tp_lora_grad_workspace_size(*args) == 0
    assert lib.tp_lora_grad_workspace_size(0, 8, 256, 4) == 0  # sums over nothing


def test_side_binding_refuses_host_tensors():
    q, s, t = torch.zeros((4, 256), dtype=torch.int8), torch.zeros(4), torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_lora_down_prequantized(q, s, torch.zeros((8, 256)))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_lora_grad_prequantized(torch.zeros((4, 16)), q, s, t, torch.zeros((16, 8)), 1.0)


# ------------------------------------------------- norm and positions of q and k
def _axes(values):
    return bytes(values)


def rp(lib, q=A, ldq=512, k=B, ldk=128, xdt=0, m=64, hq=4, hk=1, d=128, qg=C, kg=D, gdt=0, eps=1e-6, pos=E, ldp=3,
       axes=3, fr=F, ax=_axes([0] * 16 + [1] * 24 + [2] * 24), pairs=64, lay=0, qo=G, ldqo=512, ko=H, ldko=128, odt=0):
    return lib.tp_qk_norm_rope(q, ldq, k, ldk, xdt, m, hq, hk, d, qg, kg, gdt, eps, pos, ldp, axes, fr, ax, pairs, lay,
                               qo, ldqo, ko, ldko, odt, None)


ROPE_SHARED = [
    (dict(m=-1), 2), (dict(m=2 ** 31), 2), (dict(hq=-1), 2), (dict(hq=4096, hk=1), 2), (dict(hq=2 ** 40), 2),
    (dict(d=0), 2), (dict(d=12), 2), (dict(d=264), 2), (dict(pairs=6), 2), (dict(pairs=68), 2), (dict(pairs=-4), 2),
    (dict(axes=0), 2), (dict(axes=5), 2), (dict(axes=2), 13), (dict(ax=None), 1), (dict(pos=0), 1), (dict(fr=0), 1),
    (dict(ldp=2), 4), (dict(pos=E + 2), 5), (dict(fr=F + 1), 5), (dict(qg=C + 8), 5), (dict(gdt=2), 6),
    (dict(lay=2), 11), (dict(eps=0.0), 13), (dict(eps=float("nan")), 13), (dict(eps=1e-38), 13),
]


@pytest.mark.parametrize("kw,status", ROPE_SHARED + [
    (dict(q=0), 1), (dict(k=0), 1), (dict(qo=0), 1), (dict(ko=0), 1), (dict(ldq=511), 4), (dict(ldko=120), 4),
    (dict(q=A + 8), 5), (dict(ldqo=513), 5), (dict(xdt=2), 6), (dict(odt=2), 6), (dict(ldq=2 ** 62), 8),
    (dict(qo=A, odt=1), 10), (dict(qo=A + 16), 10), (dict(ko=A), 10), (dict(qo=B), 10), (dict(ko=G), 10),
    (dict(qo=C), 10), (dict(ko=E), 10), (dict(qo=F), 10),
    # views of one buffer whose columns overlap
    (dict(q=A, ldq=768, k=A + 2048 - 16, ldk=768, qo=A, ldqo=768, ko=A + 2048 - 16, ldko=768), 10),
])
def test_rope_refusals(lib, kw, status):
    assert rp(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_rope_empty_and_optional(lib):
    assert rp(lib, m=0) == 0
    assert rp(lib, hq=0, hk=0, q=0, k=0, qo=0, ko=0) == 0
    assert rp(lib, m=0, pairs=0, pos=0, fr=0, ax=None, axes=0, qg=0, kg=0, gdt=9) == 0
    # the same buffer, and column views of one buffer, are no overlap (m = 0
    # rows reach the end of the checks without a launch only if the checks pass
    # for rows too: see the refusals above for the same views one column off)
    assert rp(lib, m=0, q=A, ldq=768, k=A + 2048, ldk=768, qo=A, ldqo=768, ko=A + 2048, ldko=768) == 0


def rb(lib, yq=A, ldyq=512, yk=B, ldyk=128, ydt=0, q=I, ldq=512, k=J, ldk=128, xdt=0, m=64, hq=4, hk=1, d=128, qg=C,
       kg=D, gdt=0, eps=1e-6, pos=E, ldp=3, axes=3, fr=F, ax=_axes([0] * 16 + [1] * 24 + [2] * 24), pairs=64, lay=0,
       dq=G, lddq=512, dk=H, lddk=128, ddt=0, dqg=0xB0000000, dkg=0xC0000000, ws=0xD0000000, wsb=1 << 24):
    return lib.tp_qk_norm_rope_backward(yq, ldyq, yk, ldyk, ydt, q, ldq, k, ldk, xdt, m, hq, hk, d, qg, kg, gdt, eps,
                                        pos, ldp, axes, fr, ax, pairs, lay, dq, lddq, dk, lddk, ddt, dqg, dkg, ws, wsb,
                                        None)


@pytest.mark.parametrize("kw,status", ROPE_SHARED + [
    (dict(yq=0), 1), (dict(yk=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(dq=0), 1), (dict(dk=0), 1),
    (dict(qg=0), 1), (dict(kg=0), 1), (dict(ldyq=511), 4), (dict(ldk=120), 4), (dict(lddk=0), 4),
    (dict(yk=B + 8), 5), (dict(dqg=0xB0000002), 5), (dict(ws=0xD0000008), 5), (dict(ydt=2), 6), (dict(xdt=2), 6),
    (dict(ddt=2), 6), (dict(ws=0), 9), (dict(wsb=64), 9), (dict(ldyq=2 ** 62), 8),
    (dict(dq=A, ddt=1), 10), (dict(dq=B), 10), (dict(dk=A), 10), (dict(dq=I + 16), 10), (dict(dk=G), 10),
    (dict(dqg=G), 10), (dict(dkg=A), 10), (dict(ws=I), 10), (dict(dqg=0xC0000000), 10), (dict(ws=0xB0000000), 10),
    (dict(ws=C), 10), (dict(dqg=E), 10), (dict(dq=D), 10),
])
def test_rope_backward_refusals(lib, kw, status):
    assert rb(lib, **kw) == status, _err(lib)
    assert _err(lib)


def test_rope_backward_empty_and_workspace(lib):
    assert rb(lib, m=0, dqg=0, dkg=0, ws=0) == 0
    assert rb(lib, m=0, dqg=0, dkg=0, qg=0, kg=0, q=0, k=0, xdt=7, ws=0) == 0
    assert lib.tp_qk_norm_rope_workspace_size(64, 4, 1, 128) > 0
    for args in ((0, 4, 1, 128), (-1, 4, 1, 128), (4, -1, 1, 128), (4, 4096, 1, 128), (4, 4, 1, 12), (4, 4, 1, 264)):
        assert lib.tp_qk_norm_rope_workspace_size(*args) == 0


def test_rope_binding_refuses_host_tensors():
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_qk_norm_rope(x, x, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_qk_norm_rope_backward(x, x, None, None, 64)
