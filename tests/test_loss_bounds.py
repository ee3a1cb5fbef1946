"""The bounds of tests/loss_bounds.py hold for the arithmetic they describe and
refuse mistakes in it, planted here in a numpy copy of that arithmetic."""

import numpy as np
import pytest

from oracle import around_oracle as A
from tests import loss_bounds as L


def _case(T, d, V, seed=0):
    r = np.random.default_rng(seed)
    w = L.bf16(r.standard_normal((V, d)) * 1.5 / d ** 0.5)
    labels = r.integers(0, V, T)
    h = L.bf16(r.standard_normal((T, d)) + 2 * w[labels])
    dloss, dlse = r.standard_normal(T), 0.3 * r.standard_normal(T)
    _, _, G = A.vocab_loss_backward(h, w, labels, dloss, dlse)
    return h, w, labels, G


def _over(h, w, labels, G, gh, gw, dh_dtype, dw_dtype):
    rows = np.arange(len(labels))
    th, tw = L.bounds(G, h, w, rows, labels, L.logit_error(h, w), dh_dtype, dw_dtype)
    return (np.abs(gh - G @ w) - th).max(), (np.abs(gw - G.T @ h) - tw).max()


@pytest.mark.parametrize("T,d,V", [(100, 64, 3000), (300, 128, 2000)])
def test_bf16_outputs(T, d, V):
    h, w, labels, G = _case(T, d, V)
    rows = np.arange(T)
    hi = L.bf16(G)
    lo = np.zeros_like(G)
    lo[rows, labels] = L.bf16((G - hi)[rows, labels])
    right = hi + lo
    assert max(_over(h, w, labels, G, L.bf16(right @ w), L.bf16(right.T @ h), "bf16", "bf16")) <= 0
    # the rounding at the label left in; another row's; of the wrong sign
    shifted = np.zeros_like(G)
    shifted[rows, labels] = np.roll(lo[rows, labels], 1)
    for bad in (hi, hi + shifted, hi - lo):
        over = _over(h, w, labels, G, L.bf16(bad @ w), L.bf16(bad.T @ h), "bf16", "bf16")
        assert min(over) > 0, over


@pytest.mark.parametrize("T,d,V", [(100, 64, 300), (300, 128, 2000)])
def test_fp32_outputs(T, d, V):
    h, w, labels, G = _case(T, d, V)
    hi = L.bf16(G)
    lo = L.bf16(G - hi)
    assert max(_over(h, w, labels, G, (hi + lo) @ w, (hi + lo).T @ h, "f32", "f32")) <= 0
    rows = np.arange(T)
    one = hi.copy()
    one[rows, labels] = (hi + lo)[rows, labels]
    for bad in (hi, one, hi + np.roll(lo, 1, axis=0)):   # no second part; at the label alone; another row's
        assert min(_over(h, w, labels, G, bad @ w, bad.T @ h, "f32", "f32")) > 0
