"""moe_block_in / moe_block_out and their backward where the rows are not all
finite, against the definitions in numpy."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from oracle import around_oracle as A
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
# as in test_gpu_block.py: fp32 arithmetic relative to the terms' sizes, and a bf16 store
E, U16 = 2e-5, 2.0 ** -8


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(seed, T, d, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.exp(0.7 * torch.randn(d, generator=g)) * torch.randn((T, d), generator=g)).to(dtype)


def _values(save):
    """What a checkpoint stands for, decoded by torch."""
    T, d = save.codes.shape
    codes = save.codes.view(torch.float8_e4m3fn).float().view(T, d // 128, 128)
    return (codes * save.scales[:, :, None]).view(T, d)


# row, column: the entry that is not finite; entries of one tile, of the first and last tile of a row
BAD = [(0, 5, float("nan")), (2, 130, float("inf")), (3, 255, -float("inf")), (4, 511, float("nan"))]


def _spoil(x):
    for t, c, v in BAD:
        x[t, c] = v
    x[5, 128:256] = float("nan")   # a tile of nothing else
    bad = torch.zeros(x.shape, dtype=torch.bool)
    for t, c, _ in BAD:
        bad[t, c // 128 * 128:c // 128 * 128 + 128] = True
    bad[5, 128:256] = True
    return bad


def test_checkpoint_keeps_what_is_not_finite():
    """amax is the tile's largest size in IEEE order (NaN above all), as in the
    definition amax = max |v|: a tile that holds a NaN or an infinity decodes to
    NaN throughout (0 x inf, NaN x anything); every other tile to its own bits."""
    say("case: checkpoints of rows that are not finite")
    T, d = 7, 512
    x = _rows(1, T, d, torch.bfloat16)
    clean = A.checkpoint(x.float().numpy())
    bad = _spoil(x)
    y = _rows(2, T, d)
    ybad = _spoil(y)
    w = torch.ones(d)
    shape = moe.BlockShape(T, d)
    s_in, s_out, s_next = (moe.alloc_block_save(shape, e4m3=True) for _ in range(3))
    moe.moe_block_in(shape, x.to(DEV), w.to(DEV), save=s_in)
    finite = _rows(3, T, d, torch.bfloat16)
    xo, _ = moe.moe_block_out(shape, finite.to(DEV), y.to(DEV), w_next=w.to(DEV), save=s_out, save_next=s_next)
    for save, b in ((s_in, bad), (s_out, ybad), (s_next, ybad)):
        v = _values(save).cpu()
        assert torch.isnan(v[b]).all() and torch.isfinite(v[~b]).all()
    ok = ~bad.numpy()
    assert (s_in.codes.cpu().numpy() == clean[0])[ok].all()
    assert (s_in.scales.cpu().numpy() == clean[1])[ok[:, ::128]].all()
    # the entries themselves, where the tile's other entries are finite: x_out = x + y
    for t, c, val in BAD:
        assert float(xo[t, c]) == val or (np.isnan(val) and torch.isnan(xo[t, c]))


def test_gradients_show_what_is_not_finite():
    """Without a norm nothing but the checkpoint carries a NaN of the rows to the
    backward: dgate is NaN in the tile's columns and right in the others.  With a
    norm the whole row's dy is NaN and no other row's is."""
    say("case: backward from checkpoints of rows that are not finite")
    T, d = 7, 512
    y, do = _rows(2, T, d), _rows(4, T, d)
    bad = _spoil(y)
    gate = 0.5 * _rows(5, 1, d)
    shape = moe.BlockShape(T, d)
    x = _rows(3, T, d, torch.bfloat16)
    cols = bad.any(dim=0).numpy()
    z = np.where(np.isfinite(_np(y)), _np(y), 0)   # the columns compared hold no entry that is replaced
    for w in (None, 1 + 0.2 * _rows(6, 1, d)[0]):
        dv = None if w is None else w.to(DEV)
        for rows in (False, True):
            save = moe.alloc_block_save(shape, e4m3=True)
            moe.moe_block_out(shape, x.to(DEV), y.to(DEV), w=dv, gate=gate.to(DEV), save=save)
            dy, dw, dgate = moe.moe_block_out_backward(shape, do.to(DEV), save, w=dv, gate=gate.to(DEV),
                                                       y=y.to(DEV) if rows else None)
            if w is None:
                v = z if rows else np.where(cols, 0, _np(_values(save)))
                ref = (_np(do) * v).sum(axis=0)
                got = _np(dgate)[0]
                assert (~np.isfinite(got[cols if not rows else (~np.isfinite(_np(y))).any(axis=0)])).all()
                assert (np.abs(got - ref) <= E * np.abs(_np(do) * v).sum(axis=0))[~cols].all()
                assert torch.equal(dy.cpu(), do * gate)
            else:
                hit = bad.any(dim=1)
                assert not torch.isfinite(dy.cpu()[hit]).all(dim=1).any()
                assert torch.isfinite(dy.cpu()[~hit]).all()
                assert torch.isnan(dgate.cpu()[0, torch.from_numpy(cols)]).all()


def test_rows_that_are_not_finite_stay_alone():
    """NaN and infinities in a row reach that row's outputs only."""
    say("case: rows that are not finite beside rows that are")
    T, d = 7, 512
    x, y = _rows(1, T, d, torch.bfloat16), _rows(2, T, d)
    w = 1 + 0.2 * _rows(6, 1, d)[0]
    shape = moe.BlockShape(T, d)
    run = lambda a, b: (moe.moe_block_in(shape, a.to(DEV), w.to(DEV)),) + \
        moe.moe_block_out(shape, a.to(DEV), b.to(DEV), w=w.to(DEV), w_next=w.to(DEV))  # noqa: E731
    want = run(x, y)
    hit = _spoil(x).any(dim=1) | _spoil(y).any(dim=1)
    for a, b in zip(run(x, y), want):
        assert torch.equal(a[~hit.to(DEV)], b[~hit.to(DEV)])
        assert not torch.isfinite(a[hit.to(DEV)]).all(dim=1).any()


@pytest.mark.parametrize("T,d,gate_rows,norm,ckpt", [
    (700, 640, 90, True, True),    # gates cut into runs
    (1100, 256, 1, True, True), (1100, 72, 3, False, False),    # whole gates, several to a block
    (1100, 256, 300, True, False), (8200, 128, 100, True, True),    # up to 8 gates, and more
    (5, 8192, 0, True, True), (3, 8200, 2, True, False), (40, 4104, 7, True, False)])
def test_debug_build(T, d, gate_rows, norm, ckpt):
    """The bounds-checked build passes its checks and gives the same bits."""
    say(f"case: debug build, block ops T={T} d={d} gate_rows={gate_rows}")
    shape = moe.BlockShape(T, d, gate_rows=gate_rows)
    x, y, do = _rows(1, T, d, torch.bfloat16).to(DEV), _rows(2, T, d).to(DEV), _rows(3, T, d).to(DEV)
    w, gate = 1 + 0.1 * _rows(4, 1, d)[0].to(DEV), _rows(5, shape.gates, d).to(DEV)
    wn = w if norm else None

    def step():
        save, nxt = moe.alloc_block_save(shape, e4m3=ckpt), moe.alloc_block_save(shape, e4m3=ckpt)
        xo, nn = moe.moe_block_out(shape, x, y, w=wn, gate=gate, skip=x, w_next=w, save=save, save_next=nxt)
        n = moe.moe_block_in(shape, x, w)
        rows = {} if ckpt else dict(y=y, skip=x)
        out = moe.moe_block_out_backward(shape, do, save, w=wn, gate=gate, **rows)
        return [xo, nn, n] + [t for t in out if t is not None] + \
            list(moe.moe_block_in_backward(shape, do, w, nxt, x=None if ckpt else xo, dn_sub=do, do=do))

    a = step()
    prev = B.use_library(B.DEBUG_LIB_PATH)
    try:
        b = step()
    finally:
        B.restore_library(prev)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def _near(got, ref, size, tol=E):
    got = _np(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    over = np.abs(got - ref) - (tol * size + 2.0 ** -24 * np.abs(ref) + 1e-30)
    assert over.max(initial=-1.0) <= 0, float(over.max())


@pytest.mark.parametrize("T,d,gate_rows,norm", [
    (40, 256, None, True), (40, 256, None, False),    # no gate; neither
    (160, 256, 1, True), (1100, 128, 1, True), (1100, 128, 2, False), (1100, 128, 3, True),    # whole gates
    (33, 384, 5, True), (300, 128, 40, False), (8200, 128, 700, True), (700, 256, 30, True)])    # cut; up to 8, and more
def test_backward_from_checkpoints(T, d, gate_rows, norm):
    """Every gating, with and without a norm, from the 8-bit checkpoint."""
    say(f"case: backward from checkpoints T={T} d={d} gate_rows={gate_rows} norm={norm}")
    shape = moe.BlockShape(T, d, gate_rows=gate_rows or 0, eps=1e-5)
    x, y, do = _rows(1, T, d, torch.bfloat16), _rows(2, T, d), _rows(3, T, d)
    w = 1 + 0.2 * _rows(4, 1, d)[0] if norm else None
    gate = 0.5 * _rows(5, shape.gates, d) if gate_rows else None
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    save = moe.alloc_block_save(shape, e4m3=True)
    moe.moe_block_out(shape, dv(x), dv(y), w=dv(w), gate=dv(gate), save=save)
    dy, dw, dgate = moe.moe_block_out_backward(shape, dv(do), save, w=dv(w), gate=dv(gate))
    codes, scales, v = A.checkpoint(y.numpy())
    assert (save.codes.cpu().numpy() == codes).all() and (save.scales.cpu().numpy() == scales).all()
    r = A.rstd(_np(y), 1e-5)
    opt = lambda t: None if t is None else _np(t)  # noqa: E731
    ry, rw, rg, sy, sw, sg = A.block_out_backward(_np(do), v, opt(w), opt(gate), gate_rows or 0, r)
    _near(dy, ry, sy)
    if norm:
        _near(dw, rw, sw)
    if gate is not None:
        _near(dgate, rg, sg)
    assert (dw is None) == (w is None) and (dgate is None) == (gate is None)


def test_more_than_32768_gates():
    """32769 gates of 17 rows and one of 5, two runs of rows each: their sums take
    two launches.  dw joins 32770 partial sums: at most 16 rows, 2 runs, 513 + 18
    partial sums and the products on a path, 566 x 2^-24 = 3.4e-5 of the terms."""
    say("case: block_out backward, 32770 gates")
    T, d, L = 32769 * 17 + 5, 8, 17
    shape = moe.BlockShape(T, d, x_dtype="f32", gate_rows=L, eps=1e-5)
    x, y, do = (_rows(k, T, d) for k in (1, 2, 3))
    w, gate = 1 + 0.2 * _rows(4, 1, d)[0], 0.5 * _rows(5, shape.gates, d)
    assert shape.gates == 32770
    save = moe.alloc_block_save(shape)
    dev = [t.to(DEV) for t in (x, y, do, w, gate)]
    xo, _ = moe.moe_block_out(shape, dev[0], dev[1], w=dev[3], gate=dev[4], save=save)
    dy, dw, dgate = moe.moe_block_out_backward(shape, dev[2], save, w=dev[3], gate=dev[4], y=dev[1])
    ref, zn = A.block_out(_np(x), _np(y), None, _np(w), _np(gate), L, 1e-5, 1.0)
    _near(xo, ref, np.abs(_np(x)) + np.abs(ref - _np(x)))
    r = A.rstd(_np(y), 1e-5)
    ry, rw, rg, sy, sw, sg = A.block_out_backward(_np(do), _np(y), _np(w), _np(gate), L, r)
    _near(dy, ry, sy)
    _near(dgate, rg, sg)
    _near(dw, rw, sw, 5e-5)
