"""Pins for oracle/around_oracle.py: hand-worked values, torch autograd in
fp64, central differences, and the rules for ignored labels."""

import numpy as np
import pytest
import torch

from oracle import around_oracle as A


def _rng(seed=0):
    return np.random.default_rng(seed)


def test_block_in_by_hand():
    # mean square of (3, 4) is 12.5; with eps = 3.5 the root is 4
    n = A.block_in(np.array([[3.0, 4.0]]), np.array([2.0, 4.0]), 3.5)
    assert np.allclose(n, [[1.5, 4.0]], rtol=1e-15)


def test_block_out_by_hand():
    xo, zn = A.block_out(np.array([[1.0, -1.0]]), np.array([[4.0, 6.0]]), np.array([[1.0, 2.0]]), np.array([2.0, 4.0]),
                         np.array([[0.5, 0.25]]), 0, 3.5, 2.0)
    assert np.allclose(zn, [[1.5, 4.0]]) and np.allclose(xo, [[2.75, -1.0]])


def test_vocab_loss_by_hand():
    # logits (0, ln 3): lse = ln 4
    loss, lse, p = A.vocab_loss(np.array([[1.0]]), np.array([[0.0], [np.log(3.0)]]), np.array([1]))
    assert np.allclose(lse, np.log(4.0)) and np.allclose(loss, np.log(4.0 / 3.0)) and np.allclose(p, [[0.25, 0.75]])


@pytest.mark.parametrize("gate_rows,norm", [(0, True), (3, True), (1, True), (0, False), (3, False)])
def test_block_backward_is_autograd(gate_rows, norm):
    r, T, d, eps, beta = _rng(gate_rows + norm), 7, 12, 1e-3, 0.7
    x, y, skip, do, dn = (r.standard_normal((T, d)) for _ in range(5))
    w, wn = r.standard_normal(d), r.standard_normal(d)
    gate = r.standard_normal((-(-T // gate_rows) if gate_rows else 1, d))
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(x=x, y=y, skip=skip, w=w, wn=wn, gate=gate).items()}
    z = t["y"] - t["skip"]
    zn = z * torch.rsqrt((z * z).mean(1, keepdim=True) + eps) * t["w"] if norm else z
    rows = torch.arange(T) // (gate_rows or T)
    xo = beta * t["x"] + t["gate"][rows] * zn
    n = xo * torch.rsqrt((xo * xo).mean(1, keepdim=True) + eps) * t["wn"]
    ((xo * torch.tensor(do)).sum() + (n * torch.tensor(dn)).sum()).backward()
    # the same by the formulas: the next norm's backward gives the gradient of x_out
    xo_ = A.block_out(x, y, skip, w if norm else None, gate, gate_rows, eps, beta)[0]
    assert np.allclose(xo_, xo.detach().numpy(), rtol=1e-12)
    dxo, dwn, _, _ = A.block_in_backward(dn, None, do, xo_, wn, A.rstd(xo_, eps), 1.0)
    zz = y - skip
    dy, dw, dgate, *_ = A.block_out_backward(dxo, zz, w if norm else None, gate, gate_rows, A.rstd(zz, eps))
    assert np.allclose(dwn, t["wn"].grad, rtol=1e-10)
    assert np.allclose(dy, t["y"].grad, rtol=1e-9, atol=1e-12) and np.allclose(-dy, t["skip"].grad, atol=1e-12)
    assert np.allclose(beta * dxo, t["x"].grad, atol=1e-12) and np.allclose(dgate, t["gate"].grad, atol=1e-11)
    if norm:
        assert np.allclose(dw, t["w"].grad, atol=1e-11)


def test_vocab_loss_backward_is_autograd_and_differences():
    r, T, d, V = _rng(3), 9, 6, 11
    h, W = r.standard_normal((T, d)), r.standard_normal((V, d))
    labels = r.integers(0, V, T)
    dl, dz = r.standard_normal(T), r.standard_normal(T)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(W, requires_grad=True)
    lse = torch.logsumexp(th @ tw.t(), 1)
    loss = lse - (th @ tw.t())[torch.arange(T), torch.tensor(labels)]
    ((loss * torch.tensor(dl)).sum() + (lse * torch.tensor(dz)).sum()).backward()
    dh, dW, _ = A.vocab_loss_backward(h, W, labels, dl, dz)
    assert np.allclose(dh, th.grad, atol=1e-12) and np.allclose(dW, tw.grad, atol=1e-12)
    # central differences along a random direction of each
    f = lambda hh, ww: (lambda a, b, _: (dl * a).sum() + (dz * b).sum())(*A.vocab_loss(hh, ww, labels))  # noqa: E731
    eh, ew, e = r.standard_normal(h.shape), r.standard_normal(W.shape), 1e-5
    assert np.isclose((f(h + e * eh, W) - f(h - e * eh, W)) / (2 * e), (dh * eh).sum(), rtol=1e-7)
    assert np.isclose((f(h, W + e * ew) - f(h, W - e * ew)) / (2 * e), (dW * ew).sum(), rtol=1e-7)


def test_ignored_labels_take_no_part():
    r, T, d, V = _rng(4), 6, 5, 7
    h, W, dl = r.standard_normal((T, d)), r.standard_normal((V, d)), r.standard_normal(T)
    labels = np.array([0, -100, 6, V, -1, 3])
    bad = h.copy()
    bad[[1, 3, 4]] = np.nan
    loss, lse, _ = A.vocab_loss(bad, W, labels)
    assert (loss[[1, 3, 4]] == 0).all() and (lse[[1, 3, 4]] == 0).all() and np.isfinite(loss).all()
    dh, dW, G = A.vocab_loss_backward(bad, W, labels, dl)
    keep = [0, 2, 5]
    dh2, dW2, _ = A.vocab_loss_backward(h[keep], W, labels[keep], dl[keep])
    assert np.allclose(dh[keep], dh2) and np.allclose(dW, dW2) and (dh[[1, 3, 4]] == 0).all()
    assert np.allclose(G[keep].sum(axis=1), 0, atol=1e-15)


def test_checkpoint_values():
    v = _rng(5).standard_normal((3, 256)).astype(np.float32)
    v[1, 128:] = 0
    codes, scales, val = A.checkpoint(v)
    assert scales[1, 1] == 1 and (codes[1, 128:] == 0).all()
    for t in range(3):
        for j in range(2):
            tile = slice(128 * j, 128 * j + 128)
            q = torch.tensor(codes[t, tile]).view(torch.float8_e4m3fn).double().numpy() * float(scales[t, j])
            assert (val[t, tile] == q).all()
            # half an E4M3 step: 2^-4 of the value, or of the smallest normal number
            assert (np.abs(q - v[t, tile]) <= np.maximum(np.abs(v[t, tile]), scales[t, j] * 2.0 ** -6) * 2.0 ** -4 + 1e-7).all()
