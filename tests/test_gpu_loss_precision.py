"""The gradients of moe_vocab_loss held to the bounds of tests/loss_bounds.py:
batches of more than 64 labelled rows, every height of a row tile, several row
tiles, and several pieces of the vocabulary."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from oracle import around_oracle as A
from tests import loss_bounds as L
from tests.parity import say
from tests.test_gpu_loss import _check as _check_all
from tests.test_gpu_loss import _make, _np, _run

pytestmark = pytest.mark.gpu
DEV = "cuda"

# Rows are cut into tiles of 64 rows while the tiles fit the card, and with more
# than 128 column tiles (33100 entries: 130) into tiles of up to 256: here 64;
# 128; 192; 256 rows, and tiles of 208 and of 256 with a short last one
SIZES = [(100, 128, 300, 0.0), (770, 192, 65, 0.0), (300, 320, 2000, 0.3), (120, 64, 33100, 0.0), (180, 64, 33100, 0.0),
         (250, 64, 33100, 0.0), (600, 64, 33100, 0.1), (260, 64, 33100, 0.0), (20, 64, 3000, 0.0), (64, 320, 300, 0.0)]


def _check(args, dh_dtype, dw_dtype):
    h, w, labels, dloss, dlse = args
    _, _, dh, dw = _run(h, w, labels, dloss, dlse, dh_dtype, dw_dtype)
    hn, wn, lab = np.nan_to_num(_np(h)), _np(w), labels.numpy()
    keep = np.flatnonzero((lab >= 0) & (lab < wn.shape[0]))
    rh, rw, G = A.vocab_loss_backward(hn, wn, lab, dloss.numpy(), dlse.numpy())
    el = L.logit_error(hn[keep], wn)
    th, tw = L.bounds(G[keep], hn[keep], wn, np.arange(len(keep)), lab[keep], el, dh_dtype, dw_dtype)
    assert (np.delete(_np(dh), keep, axis=0) == 0).all()
    for name, got, ref, tol in (("dh", _np(dh)[keep], rh[keep], th), ("dw", _np(dw), rw, tw)):
        assert np.isfinite(got).all()
        over = np.abs(got - ref) - tol
        assert over.max() <= 0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("T,d,V,masked", SIZES)
def test_fp32_gradients(T, d, V, masked):
    """An fp32 gradient is not that of a bf16 operand."""
    say(f"case: vocab_loss, fp32 gradients T={T} d={d} V={V}")
    _check(_make(T + 1, T, d, V, masked), "f32", "f32")


@pytest.mark.parametrize("dh_dtype,dw_dtype", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,d,V", [(300, 192, 2000), (40, 64, 1000)])
def test_mixed_gradients(T, d, V, dh_dtype, dw_dtype):
    say(f"case: vocab_loss, dh {dh_dtype} dw {dw_dtype} T={T} d={d} V={V}")
    h, w, labels, dloss, dlse = _make(T, T, d, V, 0.1)
    _, _, dh, dw = _run(h, w, labels, dloss, dlse, dh_dtype, dw_dtype)
    # each as with both gradients of its type: bit for bit
    for k, dt in ((2, dh_dtype), (3, dw_dtype)):
        assert torch.equal((dh, dw)[k - 2], _run(h, w, labels, dloss, dlse, dt, dt)[k])


@pytest.mark.parametrize("T,d,V", [(16, 4160, 33000), (20, 4160, 33000), (20, 4160, 32700), (32, 64, 33000)])
def test_few_tokens_either_way(T, d, V):
    """Streamed or in tiles: rules on T, d and V about their edges."""
    say(f"case: vocab_loss of few tokens T={T} d={d} V={V}")
    args = _make(T, T, d, V, 0.1)
    _check_all(*args)
    _check(args, "f32", "bf16")


def _pieces(T, d, V, dtype):
    """Against float64 on the GPU, by element."""
    g = torch.Generator(device=DEV).manual_seed(3)
    w = (torch.randn((V, d), generator=g, device=DEV) * (1.5 / d ** 0.5)).bfloat16()
    h = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    labels[:2] = torch.tensor([0, V - 1])
    dl = torch.randn(T, generator=g, device=DEV)
    shape = moe.LossShape(T, d, V, dh_dtype=dtype, dw_dtype=dtype)
    _, lse = moe.moe_vocab_loss(shape, h, w, labels)
    dh, dw = moe.moe_vocab_loss_backward(shape, h, w, labels, lse, dl)
    h, w, lab, rows = h.double(), w.double(), labels.long(), torch.arange(T, device=DEV)
    G = h @ w.t()
    el = (d / 32 + 32) * 2.0 ** -24 * float((h.abs() @ w.abs().t()).max())
    G = torch.softmax(G, 1)
    G[rows, lab] -= 1
    G *= dl.double()[:, None]
    for name, got, g, b in (("dh", dh, G, w), ("dw", dw, G.t(), h)):
        ref, size = g @ b, g.abs() @ b.abs()
        tol = (4 * el + 2e-5 + L.U ** 2) * size
        if dtype == "bf16":
            r = G.clone()
            r[rows, lab] = 0
            r = r * r
            tol += 8 * L.U / 3 ** 0.5 * ((r if name == "dh" else r.t()) @ (b * b)).sqrt()
            del r
            tol += L.U * (ref.abs() + tol)
        else:
            tol += 2.0 ** -23 * ref.abs()
        over = (got.double() - ref).abs() - tol
        assert over.max() <= 0, (name, float(over.max()), int(over.argmax()) // d)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d,V", [(16384, 64, 16700), (5, 32768, 33000)])
def test_fp32_gradients_in_pieces(T, d, V):
    """Three pieces of the vocabulary (a pair of bf16 values takes twice the
    room), and two of a wide matrix."""
    say(f"case: vocab_loss in pieces, fp32 gradients T={T} d={d} V={V}")
    _pieces(T, d, V, "f32")


@pytest.mark.parametrize("T,d,V,masked", SIZES)
def test_bf16_gradients(T, d, V, masked):
    """What bf16 takes off G at a label comes back, in dh and in dw, whatever the
    number of rows."""
    say(f"case: vocab_loss, bf16 gradients T={T} d={d} V={V}")
    _check(_make(T + 1, T, d, V, masked), "bf16", "bf16")


@pytest.mark.parametrize("labels", [lambda t: 5 + 0 * t, lambda t: 512 + t % 16, lambda t: 33099 - t % 3, lambda t: 256 * (t % 9)],
                         ids=["one", "one subtile", "the last tile", "a tile's first"])
def test_bf16_gradients_of_repeated_labels(labels):
    """Many rows to one tile of the vocabulary, the other tiles none.  Labels
    repeat, so dloss has random signs and the sums are still of few terms."""
    say("case: vocab_loss, bf16 gradients of repeated labels")
    h, w, lab, dloss, dlse = _make(9, 300, 192, 33100)
    lab = labels(torch.arange(300, dtype=torch.int32)).int()
    lab[::7] = -100
    h[::7] = float("nan")
    _check((h, w, lab, dloss, dlse), "bf16", "bf16")


@pytest.mark.parametrize("T,d,V", [(16384, 64, 16700), (5, 32768, 33000)])
def test_bf16_gradients_in_pieces(T, d, V):
    """Two pieces of the vocabulary: rows whose label is in either."""
    say(f"case: vocab_loss in pieces, bf16 gradients T={T} d={d} V={V}")
    _pieces(T, d, V, "bf16")


def test_bf16_gradients_repeat_without_the_ignored():
    """Bit for bit, with and without the ignored tokens, and again."""
    say("case: vocab_loss, bf16 gradients without the ignored tokens")
    h, w, labels, dl, dz = _make(5, 900, 256, 1500, 0.6)
    keep = (labels >= 0) & (labels < 1500)
    a = _run(h, w, labels, dl, dz, "bf16", "bf16")
    b = _run(h[keep], w, labels[keep], dl[keep], dz[keep], "bf16", "bf16")
    again = _run(h, w, labels, dl, dz, "bf16", "bf16")
    assert torch.equal(a[2][keep.to(DEV)], b[2]) and torch.equal(a[3], b[3])
    assert torch.equal(a[2], again[2]) and torch.equal(a[3], again[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,masked", [(700, 192, 20000, 0.3), (17, 128, 1000, 0.0), (33, 64, 700, 0.1), (48, 192, 300, 0.0),
                                          (64, 64, 16384, 0.0), (64, 64, 17000, 0.0), (260, 64, 33100, 0.0)])
def test_gradients_debug_build(T, d, V, masked, dtype):
    """The bounds-checked build passes its checks and gives the same bits: either
    way to the logits of few tokens, and tiles of every kind."""
    say(f"case: debug build, vocab_loss with {dtype} gradients T={T} d={d} V={V}")
    args = _make(3, T, d, V, masked)
    a = _run(*args, dtype, dtype)
    prev = B.use_library(B.DEBUG_LIB_PATH)
    try:
        b = _run(*args, dtype, dtype)
    finally:
        B.restore_library(prev)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_all_of_a_large_vocabulary():
    """22100 tokens over 2^24 entries (5.7 million tiles of logits), sampled: rows
    of loss and dh, entries of dw."""
    say("case: vocab_loss, 22100 tokens over 2^24 entries")
    T, d, V = 22100, 64, 1 << 24
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.empty((V, d), dtype=torch.bfloat16, device=DEV)
    for v in range(0, V, 1 << 22):
        w[v:v + (1 << 22)] = (torch.randn((1 << 22, d), generator=g, device=DEV) * (1.5 / d ** 0.5)).bfloat16()
    h = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    labels[7] = V - 1
    dl = torch.randn(T, generator=g, device=DEV)
    shape = moe.LossShape(T, d, V, dh_dtype="bf16", dw_dtype="bf16")
    loss, lse = moe.moe_vocab_loss(shape, h, w, labels)
    dh, dw = moe.moe_vocab_loss_backward(shape, h, w, labels, lse, dl)
    # |l| <= 8 d^(1/2) 1.5 or so: products and sums of 64 terms, 2^24 exponentials joined in fp32
    rows = torch.tensor([0, 7, 8191, 16384, T - 1], device=DEV)
    hr, lab = h[rows].double(), labels[rows].long()
    el = (d / 32 + 32) * 2.0 ** -24 * float(hr.abs().sum(1).max() * w.abs().max().double())
    s, gw = torch.zeros(5, dtype=torch.float64, device=DEV), torch.zeros((5, d), dtype=torch.float64, device=DEV)
    for v in range(0, V, 1 << 21):
        p = torch.exp(hr @ w[v:v + (1 << 21)].double().t())
        s += p.sum(1)
        gw += p @ w[v:v + (1 << 21)].double()
    rz = s.log()
    rl = rz - (hr * w[lab].double()).sum(1)
    assert (lse[rows].double() - rz).abs().max() <= 2 * el + 2e-6 * (1 + float(rz.max()))
    assert (loss[rows].double() - rl).abs().max() <= 2 * el + 4e-6 * (1 + float(rz.max()))
    ref = dl[rows].double()[:, None] * (gw / s[:, None] - w[lab].double())
    size = dl[rows].abs().double()[:, None] * (float(w.abs().max()) + w[lab].abs().double())
    assert ((dh[rows].double() - ref).abs() <= L.U * ref.abs() + (4 * el + 2e-5 + 2 * L.U ** 2) * size).all()
    # dw: a label's row (that of token 7, the last entry) is -dl h but for the others' p <= e^12 / 2^24
    for t in (7, 0, 16384):
        v = int(labels[t])
        G = torch.exp(h.double() @ w[v].double() - lse.double()) * dl.double()
        G[labels.long() == v] -= dl.double()[labels.long() == v]
        ref, size = G @ h.double(), G.abs() @ h.double().abs()
        rest = torch.where(labels.long() == v, torch.zeros_like(G), G)
        tol = L.U * ref.abs() + (4 * el + 2e-5 + 2 * L.U ** 2) * size + 8 * L.U * ((rest ** 2) @ (h.double() ** 2)).sqrt()
        assert ((dw[v].double() - ref).abs() <= tol).all()
    del w, dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d,V", [(9, 128, 300), (40, 64, 20000), (300, 192, 2000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_rows_that_are_not_finite(T, d, V, dtype):
    """A NaN or an infinity in a labelled hidden row: its loss, lse and dh are NaN,
    and by the formula all of dw; every other token's results keep their bits."""
    say(f"case: vocab_loss, hidden rows not finite T={T} d={d} V={V} {dtype}")
    h, w, labels, dloss, dlse = _make(6, T, d, V)
    clean = _run(h, w, labels, dloss, dlse, dtype, dtype)
    h[3, 5], h[7, 0] = float("nan"), -float("inf")
    got = _run(h, w, labels, dloss, dlse, dtype, dtype)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[[3, 7]] = True
    for a, b in zip(got[:3], clean[:3]):
        assert torch.equal(a[~bad], b[~bad]) and torch.isfinite(a[~bad]).all()
        assert torch.isnan(a[bad]).all()
    assert torch.isnan(got[3]).all()
    # ignored, the same rows matter to nobody
    labels[[3, 7]] = -100
    got = _run(h, w, labels, dloss, dlse, dtype, dtype)
    assert all(torch.isfinite(t).all() for t in got) and (got[2][bad] == 0).all()
