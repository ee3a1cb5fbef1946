"""The roundings of moe_embed_backward's longest sums, on either side of where sums of
256 rows are formed (8192 rows).

An element of dx goes through 15 additions within its sixteen rows at most (the first
is to zero); then, below 8192 rows, through those of at most n / 16 such sums and of 15
rows behind them, or, as one of the 15 rows before, of them all: 30 + n / 16.  From 8192
on through 15 more within its 256, and of n / 256 sums, 15 of sixteen and 15 rows, or 15
each before: 60 + n / 256.  The scale and the addition to the table are one each.  Every
partial sum is at most the sum of the terms' sizes, so each rounding is at most 2^-24 of it."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from oracle import ends_oracle as A
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,first,sign", [(2100, 0, 1), (8191, 0, 1), (8191, 7, 0), (8192, 0, 1), (8192, 7, 0), (9000, 500, 1), (20000, 33, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_backward_longest_sums(T, first, sign, accumulate):
    """One token of all rows but the first few; terms of one sign, or of both."""
    say(f"case: embed backward, {T - first} of {T} rows of one token, added {accumulate}")
    g = torch.Generator().manual_seed(T + first)
    d, V = 24, 40
    dx = torch.rand((T, d), generator=g) if sign else torch.randn((T, d), generator=g)
    tok = torch.full((T,), 20, dtype=torch.int32)
    tok[:first] = torch.arange(first) % 19
    base = torch.rand((V, d), generator=g) if accumulate else None
    shape = moe.EmbedShape(T, d, V, scale=0.3)
    got = moe.moe_embed_backward(shape, tok.to(DEV), dx.to(DEV), dtable=None if base is None else base.to(DEV), accumulate=accumulate)
    f64 = lambda t: None if t is None else t.numpy().astype(np.float64)  # noqa: E731
    scale = float(np.float32(0.3))
    ref = A.embed_backward(f64(dx), tok.numpy(), V, scale, f64(base))
    mag = A.embed_magnitude(f64(dx), tok.numpy(), V, scale, f64(base))
    n = (30 + T / 16 if T < 8192 else 60 + T / 256) + 2
    err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
    say(f"  largest error {float((err / np.maximum(mag, 1e-30)).max()):.1e} of the terms' sizes, bound {n * 2.0 ** -24:.1e}")
    assert (err <= n * 2.0 ** -24 * mag).all()
