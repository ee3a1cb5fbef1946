"""CPU oracle for what stands around the layer: the norms before and after a
block with its gate and residual scale, their 8-bit checkpoints, and the
cross entropy over a vocabulary.  TEST INFRASTRUCTURE ONLY; fp64 NumPy, no
code shared with the GPU library.

    block_in    n = x r w,  r = (mean x^2 + eps)^(-1/2) per row
    block_out   z = y - skip;  zh = z r w (z without w);  x' = beta x + gate zh
    vocab_loss  l = h W^T;  lse_t = log sum_v exp l_tv;  loss_t = lse_t - l_t,label

Backward formulas are written out here and pinned against autograd and
central differences (tests/test_around_oracle.py).
"""

from __future__ import annotations

from typing import Optional

import numpy as np

from oracle.moe_oracle import e4m3_decode, e4m3_encode

F64, F32 = np.float64, np.float32


def rstd(v: np.ndarray, eps: float) -> np.ndarray:
    v = np.asarray(v, F64)
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def block_in(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    return np.asarray(x, F64) * rstd(x, eps)[:, None] * np.asarray(w, F64)


def gate_rows_of(gate: Optional[np.ndarray], T: int, d: int, gate_rows: int) -> np.ndarray:
    """The gate of every row [T, d] (ones without a gate)."""
    if gate is None:
        return np.ones((T, d))
    return np.asarray(gate, F64)[np.arange(T) // (gate_rows if gate_rows else max(T, 1))]


def block_out(x, y, skip, w, gate, gate_rows: int, eps: float, res_scale: float):
    """(x_out unrounded, zh w): the residual stream and the normed block output."""
    z = np.asarray(y, F64) - (0 if skip is None else np.asarray(skip, F64))
    zn = z if w is None else block_in(z, w, eps)
    return res_scale * np.asarray(x, F64) + gate_rows_of(gate, *z.shape, gate_rows) * zn, zn


def checkpoint(v: np.ndarray):
    """(codes, scales, the values they stand for) of fp32 rows: per 1x128 tile,
    scale = fl32(amax / 448) and codes E4M3(fl32(v * fl32(448 * fl32(1 / amax))));
    scale 1 and zero codes for a tile of zeros (amax below 2^-119)."""
    v = np.asarray(v, F32)
    T, d = v.shape
    t = v.reshape(T, d // 128, 128)
    amax = np.abs(t).max(axis=2)
    none = amax < F32(2.0 ** -119)
    nz = np.where(none, F32(1), amax)
    inv = np.where(none, F32(0), F32(448) * (F32(1) / nz)).astype(F32)
    scales = np.where(none, F32(1), nz / F32(448)).astype(F32)
    codes = e4m3_encode((t * inv[:, :, None]).astype(F32))
    val = e4m3_decode(codes).astype(F64) * scales.astype(F64)[:, :, None]
    return codes.reshape(T, d), scales, val.reshape(T, d)


def norm_backward(g, v, w, r):
    """(dv, the rows' contributions to dw, their sizes for an error bound) of
    v r w for the upstream g; v may differ from the rows r was taken from (an
    8-bit checkpoint)."""
    g, v, w = np.asarray(g, F64), np.asarray(v, F64), np.asarray(w, F64)
    vh = v * r[:, None]
    a = g * w
    dv = r[:, None] * (a - vh * (a * vh).mean(axis=1, keepdims=True))
    size = r[:, None] * (np.abs(a) + np.abs(vh) * np.abs(a * vh).mean(axis=1, keepdims=True))
    return dv, g * vh, size


def block_in_backward(dn, dn_sub, do, v, w, r, res_scale):
    """(dx, dw, |terms| of dx, |terms| of dw)."""
    g = np.asarray(dn, F64) - (0 if dn_sub is None else np.asarray(dn_sub, F64))
    dv, c, size = norm_backward(g, v, w, r)
    res = 0 if do is None else res_scale * np.asarray(do, F64)
    return dv + res, c.sum(axis=0), size + np.abs(res), np.abs(c).sum(axis=0)


def block_out_backward(do, v, w, gate, gate_rows, r):
    """(dy, dw, dgate, |terms| of each); v: the rows z (or what a checkpoint
    keeps of them), r their 1/rms (ignored without w)."""
    do, v = np.asarray(do, F64), np.asarray(v, F64)
    T, d = v.shape
    gt = gate_rows_of(gate, T, d, gate_rows)
    if w is None:
        dy, size, zh = do * gt, np.abs(do * gt), v
    else:
        dy, _, size = norm_backward(do * gt, v, w, r)
        zh = v * r[:, None]
    dw = (do * gt * zh).sum(axis=0)
    wn = np.ones(d) if w is None else np.asarray(w, F64)
    G = 1 if gate is None else gate.shape[0]
    dgate, sg = np.zeros((G, d)), np.zeros((G, d))
    which = np.arange(T) // (gate_rows if gate_rows else max(T, 1))
    np.add.at(dgate, which, do * zh * wn)
    np.add.at(sg, which, np.abs(do * zh * wn))
    return dy, dw, dgate, size, np.abs(do * gt * zh).sum(axis=0), sg


def vocab_loss(h, W, labels):
    """(loss [T], lse [T], softmax [T, V]); zeros where the label is outside [0, V)."""
    W, labels = np.asarray(W, F64), np.asarray(labels)
    T, V = len(labels), W.shape[0]
    keep = np.nonzero((labels >= 0) & (labels < V))[0]
    loss, lse, p = np.zeros(T), np.zeros(T), np.zeros((T, V))
    if len(keep):
        l = np.asarray(h, F64)[keep] @ W.T
        m = l.max(axis=1, keepdims=True)
        e = np.exp(l - m)
        lse[keep] = (m + np.log(e.sum(axis=1, keepdims=True)))[:, 0]
        loss[keep] = lse[keep] - l[np.arange(len(keep)), labels[keep]]
        p[keep] = e / e.sum(axis=1, keepdims=True)
    return loss, lse, p


def vocab_loss_backward(h, W, labels, dloss, dlse=None):
    """(dh [T, d], dW [V, d], G [T, V]): G = (dloss + dlse) softmax - dloss
    onehot, rows of ignored tokens zero (whatever h holds there)."""
    W, labels = np.asarray(W, F64), np.asarray(labels)
    _, _, p = vocab_loss(h, W, labels)
    T, V = p.shape
    dloss = np.asarray(dloss, F64)
    keep = np.nonzero((labels >= 0) & (labels < V))[0]
    G = (dloss + (0 if dlse is None else np.asarray(dlse, F64)))[:, None] * p
    G[keep, labels[keep]] -= dloss[keep]
    ignored = np.ones(T, bool)
    ignored[keep] = False
    G[ignored] = 0.0
    hk = np.asarray(h, F64)[keep]
    return G @ W, G[keep].T @ hk, G
