"""Argument checks of the entry points around the layer, on the CPU: every
call here is refused before any GPU work."""

import ctypes

import pytest

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B

FAKE = 1 << 20   # 16-byte aligned, never dereferenced
BAD = FAKE + 4


def _bs(**kw):
    return moe.BlockShape(**{**dict(T=5, d=256), **kw})


def _block_ws(shape):
    n = ctypes.c_size_t(0)
    return moe.load_library().moe_block_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), B.MOE_OK),
    (dict(T=0), B.MOE_OK),
    (dict(T=-1), B.MOE_ERR_INVALID_ARG),
    (dict(d=0), B.MOE_ERR_INVALID_ARG),
    (dict(gate_rows=-1), B.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), B.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), B.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), B.MOE_ERR_INVALID_ARG),
    (dict(res_scale=float("inf")), B.MOE_ERR_INVALID_ARG),
    (dict(x_dtype="e4m3"), B.MOE_ERR_INVALID_ARG),
    (dict(n_dtype="e4m3"), B.MOE_ERR_INVALID_ARG),
    (dict(y_dtype="e4m3"), B.MOE_ERR_INVALID_ARG),
    (dict(d=252), B.MOE_ERR_UNSUPPORTED),
    (dict(d=32776), B.MOE_ERR_UNSUPPORTED),
    (dict(d=32768), B.MOE_OK),
    (dict(T=1 << 22), B.MOE_ERR_UNSUPPORTED),
])
def test_block_shape_validation(kw, code):
    assert _block_ws(_bs(**kw))[0] == code


def test_block_workspace_covers_every_gating():
    # one row of fp32 sums per block of T / 512 rows (1 to 16); per gate where gates are longer than that
    for T, gr, rows in [(1, 0, 1), (160, 0, 160), (1024, 0, 512), (160, 1, 160), (8192, 5, 547), (20480, 0, 1280),
                        (8192, 40, 205 * 3 + 205)]:
        rc, n = _block_ws(_bs(T=T, gate_rows=gr))
        assert rc == 0 and n >= rows * 256 * 4, (T, gr, n)


def test_block_forward_refusals():
    lib, sh = moe.load_library(), _bs().c()
    r, bad = ctypes.byref, B.MOE_ERR_INVALID_ARG
    assert lib.moe_block_in(None, FAKE, FAKE, FAKE, None, None) == bad
    for args in [(None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (BAD, FAKE, FAKE), (FAKE, BAD, FAKE),
                 (FAKE, FAKE, BAD)]:
        assert lib.moe_block_in(r(sh), *args, None, None) == bad
    half = B.CBlockSave(FAKE, FAKE, None)   # codes without scales
    assert lib.moe_block_in(r(sh), FAKE, FAKE, FAKE, r(half), None) == bad
    odd = _bs(d=264).c()                    # a checkpoint takes whole 128-column tiles
    assert lib.moe_block_in(r(odd), FAKE, FAKE, FAKE, r(B.CBlockSave(FAKE, FAKE, FAKE)), None) == B.MOE_ERR_UNSUPPORTED
    out = lambda x=FAKE, y=FAKE, skip=None, w=FAKE, gate=None, wn=None, xo=FAKE, nn=None, s=None, sn=None: lib.moe_block_out(  # noqa: E731,E501
        r(sh), x, y, skip, w, gate, wn, xo, nn, s, sn, None)
    for kw in (dict(x=None), dict(y=None), dict(xo=None), dict(skip=BAD), dict(w=BAD), dict(gate=BAD),
               dict(wn=FAKE), dict(wn=BAD, nn=FAKE), dict(sn=r(B.CBlockSave(FAKE, None, None))), dict(s=r(half))):
        assert out(**kw) == bad, kw


def test_block_backward_refusals():
    lib, shape = moe.load_library(), _bs()
    sh, r, bad = shape.c(), ctypes.byref, B.MOE_ERR_INVALID_ARG
    need = _block_ws(shape)[1]
    save, empty = B.CBlockSave(FAKE, FAKE, FAKE), B.CBlockSave(FAKE, None, None)

    def b_in(dn=FAKE, sub=None, do=None, x=FAKE, w=FAKE, s=save, dx=FAKE, dw=FAKE, ws=FAKE, n=need):
        return lib.moe_block_in_backward(r(sh), dn, sub, do, x, w, None if s is None else r(s), dx, dw, ws, n, None)

    for kw in (dict(dn=None), dict(dx=None), dict(dw=None), dict(w=None), dict(sub=BAD), dict(do=BAD), dict(s=None),
               dict(s=B.CBlockSave(None, FAKE, FAKE)), dict(x=None, s=empty)):
        assert b_in(**kw) == bad, kw
    assert b_in(ws=None) == B.MOE_ERR_WORKSPACE and b_in(n=need - 1) == B.MOE_ERR_WORKSPACE

    def b_out(do=FAKE, y=FAKE, skip=None, w=FAKE, gate=FAKE, s=save, dy=FAKE, dw=FAKE, dg=FAKE, ws=FAKE, n=need):
        return lib.moe_block_out_backward(r(sh), do, y, skip, w, gate, None if s is None else r(s), dy, dw, dg, ws, n,
                                          None)

    for kw in (dict(do=None), dict(dy=None), dict(dw=None), dict(dg=None), dict(w=None), dict(gate=None), dict(s=None),
               dict(y=None, s=empty), dict(y=None, skip=FAKE), dict(skip=BAD), dict(gate=BAD), dict(y=BAD)):
        assert b_out(**kw) == bad, kw
    assert b_out(ws=None) == B.MOE_ERR_WORKSPACE and b_out(n=need - 1) == B.MOE_ERR_WORKSPACE


# ---------------------------------------------------------------- cross entropy over a vocabulary


def _loss_ws(**kw):
    shape = moe.LossShape(**{**dict(T=100, d=128, V=1000), **kw})
    f, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    rc = moe.load_library().moe_vocab_loss_workspace_size(ctypes.byref(shape.c()), ctypes.byref(f), ctypes.byref(b))
    return rc, f.value, b.value


@pytest.mark.parametrize("kw,code", [
    (dict(), B.MOE_OK),
    (dict(T=0), B.MOE_OK),
    (dict(V=1), B.MOE_OK),
    (dict(dh_dtype="bf16", dw_dtype="bf16"), B.MOE_OK),
    (dict(T=-1), B.MOE_ERR_INVALID_ARG),
    (dict(d=0), B.MOE_ERR_INVALID_ARG),
    (dict(V=0), B.MOE_ERR_INVALID_ARG),
    (dict(dh_dtype="e4m3"), B.MOE_ERR_INVALID_ARG),
    (dict(dw_dtype="e4m3"), B.MOE_ERR_INVALID_ARG),
    (dict(d=96), B.MOE_ERR_UNSUPPORTED),
    (dict(d=32832), B.MOE_ERR_UNSUPPORTED),
    (dict(V=(1 << 24) + 1), B.MOE_ERR_UNSUPPORTED),
    (dict(T=1 << 22, d=64), B.MOE_ERR_UNSUPPORTED),
    (dict(T=299_530, d=7168, V=256), B.MOE_ERR_UNSUPPORTED),   # (T + 64) d 2 reaches 2^32
    (dict(T=299_529, d=7168, V=256), B.MOE_OK),
    (dict(T=(1 << 22) - 1, d=64, V=1 << 24), B.MOE_ERR_UNSUPPORTED),   # blocks of one launch
])
def test_loss_shape_validation(kw, code):
    assert _loss_ws(**kw)[0] == code


def test_loss_workspace_keeps_no_logits():
    # T = 8192, d = 7168, V = 131072: 2 GB of bf16 logits; the backward holds a 512 MB piece,
    # the rows (117 MB) and fp32 sums of dh (235 MB, or up to 512 MB in splits)
    rc, f, b = _loss_ws(T=8192, d=7168, V=131072)
    assert rc == 0 and f < 64 << 20 and b < (512 + 112 + 512 + 1) << 20
    # G's piece is never wider than the vocabulary
    assert _loss_ws(T=1, d=64, V=256)[2] < 1 << 20


def test_loss_refusals():
    lib, shape = moe.load_library(), moe.LossShape(100, 128, 1000)
    sh, r, bad = shape.c(), ctypes.byref, B.MOE_ERR_INVALID_ARG
    _, nf, nb = _loss_ws()

    def fwd(h=FAKE, w=FAKE, lab=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, n=nf):
        return lib.moe_vocab_loss(r(sh), h, w, lab, loss, lse, ws, n, None)

    for kw in (dict(h=None), dict(h=BAD), dict(w=None), dict(w=BAD), dict(lab=None), dict(loss=None), dict(lse=None)):
        assert fwd(**kw) == bad, kw
    assert fwd(ws=None) == fwd(n=nf - 1) == fwd(ws=BAD) == B.MOE_ERR_WORKSPACE

    def bwd(h=FAKE, w=FAKE, lab=FAKE, lse=FAKE, dl=FAKE, dz=None, dh=FAKE, dw=FAKE, ws=FAKE, n=nb):
        return lib.moe_vocab_loss_backward(r(sh), h, w, lab, lse, dl, dz, dh, dw, ws, n, None)

    for kw in (dict(h=None), dict(h=BAD), dict(w=None), dict(w=BAD), dict(lab=None), dict(lse=None), dict(dl=None),
               dict(dh=None), dict(dh=BAD), dict(dw=None), dict(dw=BAD)):
        assert bwd(**kw) == bad, kw
    assert bwd(ws=None) == bwd(n=nb - 1) == bwd(ws=BAD) == B.MOE_ERR_WORKSPACE
    assert lib.moe_vocab_loss_workspace_size(r(sh), None, None) == bad
