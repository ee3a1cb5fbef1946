"""Argument checks of moe_forward_few, moe_embed* and moe_grad_*, on the CPU:
every call here is refused before any GPU work."""

import ctypes

import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B

FAKE = 1 << 20   # 16-byte aligned, never dereferenced
SUM, NORM = FAKE + (1 << 16), FAKE + (1 << 16) + 64   # the gradients' sum, their norm
BAD = FAKE + 4
INVALID, UNSUPPORTED, WORKSPACE = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
r = ctypes.byref


# ---------------------------------------------------------------- a few tokens


def _few(**kw):
    return moe.LayerShape(**{**dict(T=4, d=256, n_routed=8, n_shared=1, inter=128, top_k=2), **kw})


def _few_ws(shape):
    n = ctypes.c_size_t(0)
    return moe.load_library().moe_few_workspace_size(r(shape.c()), r(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), B.MOE_OK),
    (dict(T=0), B.MOE_OK),
    (dict(T=64), B.MOE_OK),
    (dict(T=65), UNSUPPORTED),
    (dict(T=-1), INVALID),
    (dict(d=32768), B.MOE_OK),
    (dict(d=32832), UNSUPPORTED),
    (dict(inter=32832), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED),
    (dict(d=96, inter=32, x_dtype="f32", w_dtype="f32"), B.MOE_OK),
    (dict(x_dtype="f32"), INVALID),
    (dict(w_dtype="e4m3", d=192), UNSUPPORTED),
    (dict(w_dtype="e4m3"), B.MOE_OK),
    (dict(top_k=9), INVALID),
    (dict(n_routed=16, n_groups=3, topk_groups=1), INVALID),
    (dict(n_routed=16, n_groups=4, topk_groups=2), B.MOE_OK),
])
def test_few_shape_validation(kw, code):
    assert _few_ws(_few(**kw))[0] == code


def test_few_refusals():
    lib, shape = moe.load_library(), _few()
    sh, need = shape.c(), _few_ws(shape)[1]

    def call(u=FAKE, e=FAKE, b=FAKE, w=B.Weights(*[FAKE] * 4), y=FAKE, ws=FAKE, n=need):
        return lib.moe_forward_few(r(sh), u, e, b, None if w is None else r(w), y, None, ws, n, None, None)

    for kw in (dict(u=None), dict(u=BAD), dict(e=None), dict(e=BAD), dict(b=None), dict(w=None), dict(y=None), dict(y=BAD),
               dict(w=B.Weights(FAKE, None, FAKE, FAKE)), dict(w=B.Weights(FAKE, FAKE, None, FAKE)),
               dict(w=B.Weights(FAKE, BAD, FAKE, FAKE))):
        assert call(**kw) == INVALID, kw
    assert call(ws=None) == call(ws=BAD) == call(n=need - 1) == WORKSPACE
    fp8 = _few(w_dtype="e4m3").c()
    assert lib.moe_forward_few(r(fp8), FAKE, FAKE, FAKE, r(B.Weights(*[FAKE] * 4)), FAKE, None, FAKE, 1 << 30, None,
                               None) == INVALID   # codes without scales
    assert lib.moe_few_workspace_size(r(sh), None) == INVALID
    assert lib.moe_forward_few(None, FAKE, FAKE, FAKE, r(B.Weights(*[FAKE] * 4)), FAKE, None, FAKE, need, None, None) == INVALID


def test_few_binding_checks_sizes():
    """The binding compares every tensor with the shape before it takes an address."""
    s = _few()
    u, e, b = torch.zeros(4, 256).bfloat16(), torch.zeros(8, 256).bfloat16(), torch.zeros(8)
    gu, dn = torch.zeros(8, 256, 256).bfloat16(), torch.zeros(8, 256, 128).bfloat16()
    sgu, sdn = gu[:1].clone(), dn[:1].clone()
    y, ws = torch.zeros(4, 256), torch.zeros(1 << 20, dtype=torch.uint8)
    ok = dict(u=u, centroids=e, bias=b, weights=moe.ExpertWeights(gu, dn, sgu, sdn), y=y, workspace=ws)
    for kw, word in ((dict(u=u[:3]), "u:"), (dict(centroids=e.float()), "centroids:"), (dict(bias=b[:7]), "bias:"),
                     (dict(y=y.bfloat16()), "GPU"),
                     (dict(weights=moe.ExpertWeights(gu[:7], dn, sgu, sdn)), "w_gate_up:"),
                     (dict(weights=moe.ExpertWeights(gu, dn.float(), sgu, sdn)), "w_down:"),
                     (dict(weights=moe.ExpertWeights(gu, dn, sgu, gu)), "ws_down:")):
        with pytest.raises(ValueError, match="GPU" if word == "GPU" else "GPU|" + word):
            moe.moe_forward_few(s, **{**ok, **kw})


# ---------------------------------------------------------------- the embedding


def _es(**kw):
    return moe.EmbedShape(**{**dict(T=5, d=256, V=100), **kw})


def _embed_ws(shape):
    n = ctypes.c_size_t(0)
    return moe.load_library().moe_embed_workspace_size(r(shape.c()), r(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), B.MOE_OK),
    (dict(T=0), B.MOE_OK),
    (dict(V=1), B.MOE_OK),
    (dict(V=1 << 24), B.MOE_OK),
    (dict(d=32768), B.MOE_OK),
    (dict(T=(1 << 22) - 1), B.MOE_OK),
    (dict(T=-1), INVALID),
    (dict(d=0), INVALID),
    (dict(V=0), INVALID),
    (dict(table_dtype="e4m3"), INVALID),
    (dict(x_dtype="e4m3"), INVALID),
    (dict(n_dtype="e4m3"), INVALID),
    (dict(grad_dtype="e4m3"), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(d=252), UNSUPPORTED),
    (dict(d=32776), UNSUPPORTED),
    (dict(T=1 << 22), UNSUPPORTED),
    (dict(V=(1 << 24) + 1), UNSUPPORTED),
])
def test_embed_shape_validation(kw, code):
    assert _embed_ws(_es(**kw))[0] == code


def test_embed_refusals():
    lib, sh = moe.load_library(), _es().c()

    def fwd(tok=FAKE, table=FAKE, w=FAKE, x=FAKE, n=FAKE, s=None, sh=sh):
        return lib.moe_embed(r(sh), tok, table, w, x, n, None if s is None else r(s), None)

    for kw in (dict(tok=None), dict(tok=FAKE + 2), dict(table=None), dict(table=BAD), dict(w=BAD), dict(x=None),
               dict(x=BAD), dict(n=None), dict(n=BAD), dict(w=None), dict(w=None, n=None, s=B.CBlockSave(FAKE, None, None)),
               dict(s=B.CBlockSave(FAKE, FAKE, None)), dict(s=B.CBlockSave(FAKE, BAD, FAKE))):
        assert fwd(**kw) == INVALID, kw
    odd = _es(d=264).c()   # a checkpoint takes whole 128-column tiles
    assert fwd(s=B.CBlockSave(FAKE, FAKE, FAKE), sh=odd) == UNSUPPORTED
    need = _embed_ws(_es())[1]

    def bwd(tok=FAKE, dx=FAKE, dt=FAKE, acc=0, ws=FAKE, n=need):
        return lib.moe_embed_backward(r(sh), tok, dx, dt, acc, ws, n, None)

    for kw in (dict(tok=None), dict(tok=FAKE + 1), dict(dx=None), dict(dx=BAD), dict(dt=None), dict(dt=BAD)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(ws=None) == bwd(ws=BAD) == bwd(n=need - 1) == WORKSPACE
    with pytest.raises(ValueError, match="no dtable"):
        moe.moe_embed_backward(_es(), torch.zeros(5, dtype=torch.int32), torch.zeros(5, 256), accumulate=True)


# ---------------------------------------------------------------- gradients


def _tensors(*ts):
    return (B.CTensor * max(len(ts), 1))(*ts)


def test_grad_workspace():
    n = ctypes.c_size_t(0)
    lib = moe.load_library()
    sizes = []
    for k in (0, 1, 112, 113, 1000):
        assert lib.moe_grad_workspace_size(k, r(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[2] < sizes[3]
    assert lib.moe_grad_workspace_size(-1, r(n)) == INVALID and lib.moe_grad_workspace_size(1, None) == INVALID


@pytest.mark.parametrize("ts", [
    [(None, 5, B.F32)],                                           # no address
    [(FAKE, -1, B.F32)],
    [(FAKE, 5, B.E4M3)],
    [(FAKE + 2, 5, B.F32)],                                       # not an element's address
    [(FAKE + 1, 5, B.BF16)],
    [(FAKE, 5, B.F32), (FAKE, 5, B.F32)],                         # the same twice
    [(FAKE, 5, B.F32), (FAKE + 64, 5, B.F32), (FAKE + 16, 1, B.F32)],   # the last element of the first
    [(FAKE, 5, B.BF16), (FAKE + 8, 2, B.BF16)],
])
def test_grad_refuses_tensors(ts):
    lib, c = moe.load_library(), _tensors(*ts)
    assert lib.moe_grad_sumsq(c, len(ts), SUM, FAKE, 1 << 20, None) == INVALID
    assert lib.moe_grad_clip(c, None, len(ts), SUM, 1.0, NORM, None) == INVALID


def test_grad_refusals():
    lib = moe.load_library()
    two = _tensors((FAKE, 5, B.F32), (FAKE + 20, 5, B.F32))
    need = 1 << 20
    assert lib.moe_grad_sumsq(None, 1, SUM, FAKE, need, None) == INVALID
    assert lib.moe_grad_sumsq(two, -1, SUM, FAKE, need, None) == INVALID
    assert lib.moe_grad_sumsq(two, 2, None, FAKE, need, None) == INVALID
    assert lib.moe_grad_sumsq(two, 2, BAD, FAKE, need, None) == INVALID
    assert lib.moe_grad_sumsq(two, 2, SUM, None, need, None) == WORKSPACE
    assert lib.moe_grad_sumsq(two, 2, SUM, FAKE, 100, None) == WORKSPACE
    for m in (0.0, -1.0, float("nan")):
        assert lib.moe_grad_clip(two, None, 2, SUM, m, NORM, None) == INVALID
    assert lib.moe_grad_clip(two, None, 2, None, 1.0, NORM, None) == INVALID
    assert lib.moe_grad_clip(two, None, 2, SUM, 1.0, NORM + 2, None) == INVALID
    # outputs: another size, over an input that is not theirs, over each other, in place in another type
    for out in ([(FAKE + 400, 5, B.F32), (FAKE + 800, 4, B.F32)], [(FAKE + 20, 5, B.F32), (FAKE, 5, B.F32)],
                [(FAKE + 400, 5, B.F32), (FAKE + 404, 5, B.F32)], [(FAKE, 5, B.BF16), (FAKE + 20, 5, B.F32)],
                [(None, 5, B.F32), (FAKE + 20, 5, B.F32)]):
        assert lib.moe_grad_clip(two, _tensors(*out), 2, SUM, 1.0, NORM, None) == INVALID, out
    huge = _tensors((FAKE, (1 << 44) + 1, B.BF16))
    assert lib.moe_grad_sumsq(huge, 1, SUM, FAKE, need, None) == UNSUPPORTED
    # the sum or the norm in a tensor, or in each other
    assert lib.moe_grad_sumsq(two, 2, FAKE + 16, FAKE, need, None) == INVALID
    for at, norm in ((FAKE + 32, NORM), (SUM, FAKE + 36), (SUM, SUM), (SUM, SUM + 4)):
        assert lib.moe_grad_clip(two, None, 2, at, 1.0, norm, None) == INVALID, (at, norm)
    assert lib.moe_grad_clip(None, None, 0, SUM, 1.0, SUM + 4, None) == INVALID


def test_tensor_list_refuses():
    with pytest.raises(ValueError, match="f32 or bf16"):
        moe.TensorList([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError, match="GPU"):
        moe.TensorList([torch.zeros(3)])


# ---------------------------------------------------------------- devices


def _compared(monkeypatch, fn):
    """The tensors whose devices a call compares before it takes their addresses (which host tensors do not have)."""
    seen = []
    monkeypatch.setattr(B, "_same_device", lambda *ts: seen.extend(id(t) for t in ts if t is not None))
    with pytest.raises(ValueError, match="GPU"):
        fn()
    return seen


@pytest.mark.parametrize("w_dtype", ["bf16", "e4m3"])
def test_few_compares_every_device(monkeypatch, w_dtype):
    s = _few(w_dtype=w_dtype)
    code = torch.uint8 if w_dtype == "e4m3" else torch.bfloat16
    w = [torch.zeros(n, dtype=code) for n in ((8, 256, 256), (8, 256, 128), (1, 256, 256), (1, 256, 128))]
    if w_dtype == "e4m3":
        w += [torch.zeros(n) for n in ((8, 2, 2), (8, 2, 1), (1, 2, 2), (1, 2, 1))]
    rest = dict(u=torch.zeros(4, 256).bfloat16(), centroids=torch.zeros(8, 256).bfloat16(), bias=torch.zeros(8),
                y=torch.zeros(4, 256), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    seen = _compared(monkeypatch, lambda: moe.moe_forward_few(s, weights=moe.ExpertWeights(*w), **rest))
    assert {id(t) for t in [*w, *rest.values()]} <= set(seen)


def test_embed_compares_every_device(monkeypatch):
    s = _es()
    args = dict(tokens=torch.zeros(5, dtype=torch.int32), table=torch.zeros(100, 256), w_next=torch.zeros(256),
                x=torch.zeros(5, 256), n_next=torch.zeros(5, 256).bfloat16())
    save = [torch.zeros(5), torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(5, 2)]
    seen = _compared(monkeypatch, lambda: moe.moe_embed(s, save_next=moe.BlockSave(*save), **args))
    assert {id(t) for t in [*args.values(), *save]} <= set(seen)


def test_other_calls_compare_every_device(monkeypatch):
    tokens, dx = torch.zeros(5, dtype=torch.int32), torch.zeros(5, 256)
    dt, ws = torch.zeros(100, 256), torch.zeros(1 << 20, dtype=torch.uint8)
    seen = _compared(monkeypatch, lambda: moe.moe_embed_backward(_es(), tokens, dx, dtable=dt, workspace=ws))
    assert {id(t) for t in (tokens, dx, dt, ws)} <= set(seen)
    sumsq, norm = torch.zeros(1, dtype=torch.float64), torch.zeros(1)
    assert {id(sumsq), id(ws)} <= set(_compared(monkeypatch, lambda: moe.moe_grad_sumsq([], sumsq=sumsq, workspace=ws)))
    assert {id(sumsq), id(norm)} <= set(_compared(monkeypatch, lambda: moe.moe_grad_clip([], sumsq, 1.0, norm=norm)))
