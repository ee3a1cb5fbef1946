"""moe_vocab_loss and its backward on the GPU against the fp64 oracle.

Tolerances.  bf16 products are exact in fp32; a logit adds them in d / 32 MFMA
steps of 32, so its error is at most EL = (d / 32 + 32) 2^-24 sum_k |h_k w_k|.
loss and lse: 2 max_v EL plus 2e-6 of their size and of the sum's (a hardware
exponential, at most V / 4096 + 80 additions on a path, 131073 / 4096 here).
dh, dw: G is rounded to bf16 once, an error of at most 2^-8 |G_tv| with
independent signs, so of standard deviation at most 2^-8 / sqrt(3) sqrt(sum G^2 W^2)
in a sum; eight of them are allowed, plus the rounding of a bf16 output (2^-8),
plus (4 max EL + 2e-5) sum |G||W| for the recomputed logits and the fp32 sums.
"""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from oracle import around_oracle as A
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U16 = 2.0 ** -8


def _make(seed, T, d, V, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((V, d), generator=g) * (1.5 / d ** 0.5)).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    h = (torch.randn((T, d), generator=g) + 2.0 * w[labels.long()].float()).bfloat16()
    drop = torch.rand(T, generator=g) < masked
    labels[drop] = torch.where(torch.arange(T, dtype=torch.int32)[drop] % 2 == 0, -100, V).int()
    h[drop] = float("nan")
    return h, w, labels, torch.randn(T, generator=g), 0.3 * torch.randn(T, generator=g)


def _run(h, w, labels, dloss, dlse, dh_dtype="f32", dw_dtype="f32"):
    T, d = h.shape
    shape = moe.LossShape(T, d, w.shape[0], dh_dtype=dh_dtype, dw_dtype=dw_dtype)
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    h, w, labels = dv(h), dv(w), dv(labels)
    loss, lse = moe.moe_vocab_loss(shape, h, w, labels)
    dh, dw = moe.moe_vocab_loss_backward(shape, h, w, labels, lse, dv(dloss), dv(dlse))
    torch.cuda.synchronize()
    return loss, lse, dh, dw


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(h, w, labels, dloss, dlse, dh_dtype="f32", dw_dtype="f32"):
    loss, lse, dh, dw = _run(h, w, labels, dloss, dlse, dh_dtype, dw_dtype)
    hn, wn, lab = np.nan_to_num(_np(h)), _np(w), labels.numpy()
    d = hn.shape[1]
    keep = (lab >= 0) & (lab < wn.shape[0])
    rl, rz, _ = A.vocab_loss(hn, wn, lab)
    rh, rw, G = A.vocab_loss_backward(hn, wn, lab, dloss.numpy(), None if dlse is None else dlse.numpy())
    el = (d / 32 + 32) * 2.0 ** -24 * (np.abs(hn) @ np.abs(wn).T).max(axis=1)
    top = float(el[keep].max(initial=0))
    for got, ref in ((_np(loss), rl), (_np(lse), rz)):
        assert (got[~keep] == 0).all()
        over = np.abs(got - ref) - (2 * el + 2e-6 * (1 + np.abs(ref) + np.abs(rz)))
        assert over[keep].max(initial=-1) <= 0, over[keep].max()
    for got, ref, a, b, dt in ((_np(dh), rh, G, wn, dh_dtype), (_np(dw), rw, G[keep].T, hn[keep], dw_dtype)):
        assert np.isfinite(got).all()
        tol = 8 * U16 / 3 ** 0.5 * np.sqrt((a * a) @ (b * b)) + (4 * top + 2e-5) * (np.abs(a) @ np.abs(b))
        tol += (U16 if dt == "bf16" else 2.0 ** -24) * np.abs(ref)
        over = np.abs(got - ref) - tol
        assert over.max(initial=-1) <= 1e-30, (over.max(), np.abs(ref).max())
    assert (_np(dh)[~keep] == 0).all()


# one token; vocabularies of one entry, about a tile's 64 and 256 and not
# multiples of anything; row counts about the 16-row subtiles, the 64-row steps
# and the 256-row tiles; few tokens on either forward (up to 64 with at most
# 16384 entries, and more entries than that)
SIZES = [(1, 64, 1), (1, 64, 256), (3, 128, 257), (15, 64, 1000), (17, 192, 255), (33, 2048, 300), (48, 64, 65),
         (64, 320, 191), (50, 64, 16700), (100, 128, 300), (200, 64, 520), (256, 256, 512), (257, 320, 777),
         (300, 512, 4099), (513, 64, 300), (770, 192, 65), (40, 7168, 600)]


@pytest.mark.parametrize("T,d,V", SIZES)
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_loss(T, d, V, masked):
    say(f"case: vocab_loss T={T} d={d} V={V} masked={masked}")
    h, w, labels, dl, dz = _make(T + d, T, d, V, masked)
    _check(h, w, labels, dl, dz if T % 2 else None, "f32" if T % 3 else "bf16", "bf16" if d % 128 else "f32")


def test_all_tokens_ignored():
    say("case: vocab_loss, every token ignored")
    h, w, labels, dl, _ = _make(0, 70, 128, 300)
    labels[:] = -100
    h[:] = float("nan")
    loss, lse, dh, dw = _run(h, w, labels, dl, None)
    for t in (loss, lse, dh, dw):
        assert (t == 0).all()


def test_no_tokens():
    say("case: vocab_loss of no tokens")
    e = torch.empty(0)
    loss, lse, dh, dw = _run(torch.empty((0, 64)).bfloat16(), torch.ones((300, 64)).bfloat16(), e.int(), e, None)
    assert loss.shape == (0,) and dh.shape == (0, 64) and (dw == 0).all()


def test_masked_tokens_change_nothing():
    """The kept tokens' results are those of a batch without the others, bit for bit."""
    say("case: vocab_loss with and without its masked tokens")
    h, w, labels, dl, dz = _make(5, 900, 256, 1500, 0.6)
    keep = (labels >= 0) & (labels < 1500)
    a = _run(h, w, labels, dl, dz)
    b = _run(h[keep], w, labels[keep], dl[keep], dz[keep])
    for k in range(3):
        assert torch.equal(a[k][keep.to(DEV)], b[k]) and (a[k][~keep.to(DEV)] == 0).all()
    assert torch.equal(a[3], b[3])


def test_extreme_logits():
    """Logits of +-2e4 (one entry takes all the weight) and identical rows."""
    say("case: vocab_loss, extreme logits")
    T, d, V = 20, 64, 520
    h = torch.zeros((T, d)).bfloat16()
    w = torch.zeros((V, d)).bfloat16()
    h[:, 0] = 200.0
    w[3, 0], w[300, 0] = 100.0, -100.0
    labels = torch.full((T,), 3, dtype=torch.int32)
    labels[1], labels[2] = 300, 7
    loss, lse, dh, dw = _run(h, w, labels, torch.ones(T), None)
    assert (lse == 20000.0).all()
    assert loss[0] == 0 and loss[1] == 40000.0 and loss[2] == 20000.0
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
    assert dh[1, 0] == 200.0 and dh[0].abs().max() == 0
    # equal logits: loss = log V
    loss, *_ = _run(torch.zeros((T, d)).bfloat16(), w, labels, torch.ones(T), None)
    assert torch.allclose(loss, torch.full((T,), float(np.log(V)), device=DEV), rtol=1e-6, atol=0)


def test_large_vocabulary_one_token():
    say("case: vocab_loss of 2 tokens over 131073 entries")
    h, w, labels, dl, dz = _make(6, 2, 64, 131073)
    labels[1] = 131072   # the one entry of the last tile
    h[1] = (2.0 * w[131072].float()).bfloat16()
    _check(h, w, labels, dl, dz, "bf16", "bf16")


def _reference_on_gpu(h, w, labels, dl):
    lab = labels.long()
    logits = h.double() @ w.double().t()
    lse = torch.logsumexp(logits, 1)
    loss = lse - logits.gather(1, lab[:, None])[:, 0]
    G = torch.exp(logits - lse[:, None])
    G[torch.arange(len(lab), device=DEV), lab] -= 1
    G *= dl.double()[:, None]
    return loss, lse, G @ w.double(), G.t() @ h.double()


@pytest.mark.parametrize("T,d,V", [(16384, 64, 16700), (5, 32768, 33000)])
def test_pieces_of_the_vocabulary(T, d, V):
    """More than one piece: a long batch, and a wide matrix.  Normwise: one
    rounding of G (2^-8 at most) and one of a bf16 output, so at most 1e-2."""
    say(f"case: vocab_loss in pieces T={T} d={d} V={V}")
    g = torch.Generator(device=DEV).manual_seed(1)
    w = (torch.randn((V, d), generator=g, device=DEV) * (1.5 / d ** 0.5)).bfloat16()
    h = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    labels[:2] = torch.tensor([0, V - 1])
    dl = torch.randn(T, generator=g, device=DEV)
    shape = moe.LossShape(T, d, V, dh_dtype="bf16", dw_dtype="bf16")
    loss, lse = moe.moe_vocab_loss(shape, h, w, labels)
    dh, dw = moe.moe_vocab_loss_backward(shape, h, w, labels, lse, dl)
    rl, rz, rh, rw = _reference_on_gpu(h, w, labels, dl)
    el = (d / 32 + 32) * 2.0 ** -24 * float(h.float().norm(dim=1).max() * w.float().norm(dim=1).max())
    assert (loss.double() - rl).abs().max() <= 2 * el + 2e-5 and (lse.double() - rz).abs().max() <= 2 * el + 2e-5
    for got, ref in ((dh, rh), (dw, rw)):
        # by blocks of rows, so that an error in one piece cannot hide
        for r0 in range(0, ref.shape[0], 4096):
            a, b = got[r0:r0 + 4096].double(), ref[r0:r0 + 4096]
            assert (a - b).norm() <= 1e-2 * b.norm(), (r0, float((a - b).norm() / b.norm()))
    del w, h, dh, dw, rh, rw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d,V,masked", [(1, 256, 4099, 0.0), (2, 64, 1000, 0.0), (5, 128, 700, 0.5), (17, 320, 2000, 0.0),
                                          (64, 64, 4099, 0.0), (65, 128, 520, 0.2), (300, 64, 2000, 0.85)])
def test_gradients_of_few_rows(T, d, V, masked):
    """Up to 64 rows: dw carries G's rounding errors too, which are themselves
    rounded (2^-9 of 2^-9 of an element); dh that of the label's element."""
    say(f"case: vocab_loss, few rows T={T} d={d} V={V} masked={masked}")
    h, w, labels, dloss, dlse = _make(T, T, d, V, masked)
    _, _, dh, dw = _run(h, w, labels, dloss, dlse)
    hn, wn, lab = np.nan_to_num(_np(h)), _np(w), labels.numpy()
    keep = np.flatnonzero((lab >= 0) & (lab < V))
    assert len(keep) <= 64
    rh, rw, G = A.vocab_loss_backward(hn, wn, lab, dloss.numpy(), dlse.numpy())
    top = (d / 32 + 32) * 2.0 ** -24 * (np.abs(hn) @ np.abs(wn).T)[keep].max(initial=0)
    rest = G.copy()
    rest[keep, lab[keep]] = 0
    tol = 8 * U16 / 3 ** 0.5 * np.sqrt((rest * rest) @ (wn * wn)) + (4 * top + 2e-5) * (np.abs(G) @ np.abs(wn))
    over = np.abs(_np(dh) - rh) - tol - 2.0 ** -23 * np.abs(rh)
    assert over.max() <= 1e-30, over.max()
    over = np.abs(_np(dw) - rw) - (4 * top + 2e-5 + 2.0 ** -17) * (np.abs(G).T @ np.abs(hn)) - 2.0 ** -23 * np.abs(rw)
    assert over.max() <= 1e-30, over.max()


def test_equal_weights_do_not_bias_the_gradient():
    """dloss = 1 / T, 0.2% from a bf16 value: G is held over its mantissa, so the
    label's element (p - 1, here p below 1/2) is off by at most p and 2^-9 of the
    weight, another by 2^-9 of itself."""
    say("case: vocab_loss, equal weights")
    T, d, V = 300, 128, 2000
    g = torch.Generator().manual_seed(5)
    w = (torch.randn((V, d), generator=g) * (1.0 / d ** 0.5)).bfloat16()
    h = torch.randn((T, d), generator=g).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    dloss = torch.full((T,), 1 / T)
    _, _, dh, dw = _run(h, w, labels, dloss, None)
    hn, wn, lab, t = _np(h), _np(w), labels.numpy(), np.arange(T)
    rh, rw, G = A.vocab_loss_backward(hn, wn, lab, dloss.numpy())
    p = G[t, lab] * T + 1
    assert 0 < p.min() and p.max() < 0.5
    err = 2.0 ** -9 * np.abs(G)
    err[t, lab] = np.minimum(p, 2.0 ** -9) / T
    top = (d / 32 + 32) * 2.0 ** -24 * (np.abs(hn) @ np.abs(wn).T).max()
    for got, ref, e, a, b in ((_np(dh), rh, err, G, wn), (_np(dw), rw, err.T, G.T, hn)):
        over = np.abs(got - ref) - e @ np.abs(b) - (4 * top + 2e-5) * (np.abs(a) @ np.abs(b)) - 2.0 ** -23 * np.abs(ref)
        assert over.max() <= 1e-30, over.max()


def test_weights_that_are_not_finite():
    """A row whose dloss is NaN or infinite leaves the other rows' dh as they are."""
    say("case: vocab_loss, dloss not finite")
    h, w, labels, dloss, _ = _make(6, 9, 128, 300)
    clean = _run(h, w, labels, dloss, None)[2]
    dloss[3], dloss[7] = float("nan"), float("inf")
    dh = _run(h, w, labels, dloss, None)[2]
    others = [t for t in range(9) if t not in (3, 7)]
    # (the scale may be another's mantissa: the rounding of G differs, 2^-8 of a row's sums each)
    tol = 2 * U16 * (dloss[others].abs()[:, None] * 2 * w.float().abs().max(dim=0).values)
    assert ((dh - clean)[others].cpu().abs() <= tol).all()
    assert not torch.isfinite(dh[3]).any() and not torch.isfinite(dh[7]).any()


def test_gradient_is_the_difference_quotient():
    """Along random directions of h and w, against central differences of the
    GPU's own loss in steps that bf16 holds exactly.  Errors: the loss's own
    (2e-5 each) over the step, the third-order term, and the bf16 rounding of
    G (2^-8 of the terms' sizes at most, of random sign)."""
    say("case: vocab_loss against differences")
    T, d, V, e = 64, 128, 500, 2.0 ** -5
    g = torch.Generator().manual_seed(2)
    # multiples of 1/32 below 4: adding or taking 1/32 stays exact in bf16's 8 bits
    h = (torch.randint(-60, 61, (T, d), generator=g).float() / 32).bfloat16()
    w = (torch.randint(-30, 31, (V, d), generator=g).float() / 256).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    dl, dz = torch.randn(T, generator=g), 0.5 * torch.randn(T, generator=g)
    loss, lse, dh, dw = _run(h, w, labels, dl, dz)

    def f(h, w):
        shape = moe.LossShape(T, d, V)
        loss, lse = moe.moe_vocab_loss(shape, h.to(DEV), w.to(DEV), labels.to(DEV))
        return float((loss.double().cpu() * dl.double()).sum() + (lse.double().cpu() * dz.double()).sum())

    for k in range(3):
        s = torch.where(torch.rand((T, d), generator=g) < 0.1, 1.0, 0.0) * torch.sign(torch.randn((T, d), generator=g))
        hp, hm = (h.float() + e * s).bfloat16(), (h.float() - e * s).bfloat16()
        assert torch.equal(hp.float() - h.float(), e * s) and torch.equal(h.float() - hm.float(), e * s)
        num = (f(hp, w) - f(hm, w)) / (2 * e)
        ana = float((dh.cpu().double() * s.double()).sum())
        scale = float((dh.cpu().double().abs() * s.double().abs()).sum())
        assert abs(num - ana) <= 2e-5 * T / e + 2e-2 * scale, (num, ana, scale)
        q = 2.0 ** -8
        s = torch.where(torch.rand((V, d), generator=g) < 0.1, 1.0, 0.0) * torch.sign(torch.randn((V, d), generator=g))
        wp, wm = (w.float() + q * s).bfloat16(), (w.float() - q * s).bfloat16()
        assert torch.equal(wp.float() - w.float(), q * s) and torch.equal(w.float() - wm.float(), q * s)
        num = (f(h, wp) - f(h, wm)) / (2 * q)
        ana = float((dw.cpu().double() * s.double()).sum())
        scale = float((dw.cpu().double().abs() * s.double().abs()).sum())
        assert abs(num - ana) <= 2e-5 * T / q + 2e-2 * scale, (num, ana, scale)


def test_loss_repeats_and_graph():
    """Bit-identical repeats, on a side stream, and replayed from a captured graph."""
    say("case: vocab_loss repeats and graph")
    h, w, labels, dl, dz = (t.to(DEV) for t in _make(7, 333, 256, 2000, 0.2))
    shape = moe.LossShape(333, 256, 2000)
    wf = torch.empty(moe.loss_workspace_size(shape), dtype=torch.uint8, device=DEV)
    wb = torch.empty(moe.loss_workspace_size(shape, True), dtype=torch.uint8, device=DEV)

    def step():
        loss, lse = moe.moe_vocab_loss(shape, h, w, labels, workspace=wf)
        return (loss, lse) + moe.moe_vocab_loss_backward(shape, h, w, labels, lse, dl, dz, workspace=wb)

    first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = step()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, out):
            assert torch.equal(a, b)
        again = step()
        torch.cuda.synchronize()
        assert torch.equal(again[3], first[3])


def test_loss_binding_refuses():
    h, w, labels, dl, _ = (t.to(DEV) for t in _make(8, 4, 64, 100))
    shape = moe.LossShape(4, 64, 100)
    with pytest.raises(ValueError):
        moe.moe_vocab_loss(shape, h, w, labels.long())          # int32 labels
    with pytest.raises(ValueError):
        moe.moe_vocab_loss(shape, h.float(), w, labels)
    with pytest.raises(ValueError):
        moe.moe_vocab_loss(shape, h, w[:99], labels)
    with pytest.raises(ValueError):
        moe.moe_vocab_loss(shape, h, w.t().contiguous().t(), labels)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_vocab_loss(shape, h, w, labels, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("T,d,V,masked", [(7, 128, 300, 0.3), (100, 192, 777, 0.3), (600, 512, 20000, 0.5),
                                          (4096, 256, 2000, 0.1)])
def test_loss_debug_build(T, d, V, masked):
    """The bounds-checked build passes its index checks and gives the same bits."""
    say(f"case: debug build, vocab_loss T={T} d={d} V={V}")
    args = _make(T, T, d, V, masked)
    a = _run(*args)
    prev = B.use_library(B.DEBUG_LIB_PATH)
    try:
        b = _run(*args)
    finally:
        B.restore_library(prev)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
