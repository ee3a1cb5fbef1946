"""The example model's two ends and its scoring, run together: the embedding and
its gradient, the clipping of a step's gradients, single tokens and small batches
through the layer's forward for a few tokens."""

import numpy as np
import pytest
import torch

from mixture_experts_layer_deepseekmoe_amd import binding as moe
from mixture_experts_layer_deepseekmoe_amd import example as X
from oracle import ends_oracle as A
from tests.parity import say

pytestmark = pytest.mark.gpu
SMALL = X.ModelShape(T=96, d=128, layers=2, vocab=200, n_routed=8, inter=64, top_k=2)


def test_the_embedding_is_the_table_and_its_norm():
    """x and n of the first block, bit for bit: fp32 rows unscaled, and moe_block_in of them."""
    say("case: example, embedding")
    model = X.Model(SMALL, seed=2)
    tokens, _ = X.make_batch(SMALL, 1)
    x, n = moe.moe_embed(SMALL.embed(), tokens, model.params["embed"], w_next=model.params["0.w_in"])
    assert torch.equal(x, model.params["embed"][tokens.long()])
    assert torch.equal(n, moe.moe_block_in(SMALL.block(), x, model.params["0.w_in"]))


def test_a_step_repeats_and_is_clipped_together():
    """Two runs of a step give the same bits, the embedding's gradient among them; the
    clipped gradients are the step's, scaled by the limit over their norm."""
    say("case: example, a step's gradients, twice, clipped")
    model = X.Model(SMALL, seed=3)
    batch = X.make_batch(SMALL, 7)
    _, g1 = model.step(*batch)
    _, g2 = model.step(*batch)
    assert all(torch.equal(g1[k], g2[k]) for k in g1)
    ref = {k: v.double().cpu().numpy() for k, v in g1.items()}
    norm = np.sqrt(A.sumsq(ref.values()))
    got = X.clip(g2, 0.5 * norm)
    assert abs(float(got) - norm) <= 2.0 ** -23 * norm
    for k, v in g2.items():   # a product in 64 bits, rounded to fp32
        assert np.abs(v.double().cpu().numpy() - 0.5 * ref[k]).max() <= 1.01 * 2.0 ** -24 * np.abs(0.5 * ref[k]).max(), k
    got = X.clip(g1, 2 * norm)
    assert abs(float(got) - norm) <= 2.0 ** -23 * norm
    assert all(np.array_equal(g1[k].double().cpu().numpy(), ref[k]) for k in g1)


@pytest.mark.parametrize("T", [1, 5, 64])
def test_scoring_few_tokens(T):
    """A few tokens score as the same tokens within a batch that moe_forward takes.
    Each layer's y differs by moe_forward's roundings of H and Y, 2 x 2^-9 of the experts'
    part, the rows between by theirs, 2^-9 (bf16): over two layers and the final norm at
    most 8 x 2^-9 of a row h, normwise, so a logit by that times |h| |w| and a loss, the
    difference of two such, by twice it: |h| = sqrt(d), |w| about 1."""
    say(f"case: example, scoring {T} tokens")
    model = X.Model(SMALL, seed=4)
    tokens, labels = X.make_batch(SMALL, 9, ignored=0.0)
    all_of_them = model.loss(tokens, labels)
    assert SMALL.T > moe.FEW_TOKENS
    few = model.loss(tokens[:T].contiguous(), labels[:T].contiguous())
    w = float(model.params["w_vocab"].norm(dim=1).max())
    assert float((few - all_of_them[:T]).abs().max()) <= 2 * 8 * 2.0 ** -9 * np.sqrt(SMALL.d) * w


def test_training_with_a_limit_runs():
    say("case: example, training with clipped gradients")
    lines = []
    model = X.train(SMALL, 3, max_norm=0.01, log=lines.append)
    assert len(lines) == 2 and all(bool(torch.isfinite(p).all()) for p in model.params.values())
