"""The example model at the edges of what it takes: tokens of other types, devices and
strides, wide experts, training steps whose gradients are not finite."""

import pytest
import torch

from mixture_experts_layer_deepseekmoe_amd import binding as moe
from mixture_experts_layer_deepseekmoe_amd import example as X
from tests.parity import say

pytestmark = pytest.mark.gpu
SMALL = X.ModelShape(T=96, d=128, layers=2, vocab=200, n_routed=8, inter=64, top_k=2)


@pytest.mark.parametrize("T", [3, 96])
def test_tokens_of_any_integer_type(T):
    """int64, int16, strided and host tokens score as the same int32 ones, bit for bit;
    values that int32 does not hold are outside the vocabulary."""
    say(f"case: example, token types, {T} tokens")
    model = X.Model(SMALL, seed=5)
    tokens, labels = (t[:T].contiguous() for t in X.make_batch(SMALL, 3))
    want = model.loss(tokens, labels)
    strided = torch.stack([tokens, tokens + 1], 1)[:, 0]
    assert not strided.is_contiguous() or T == 1
    for t in (tokens.long(), tokens.short(), strided, strided.long(), tokens.cpu(), tokens.cpu().long()):
        assert torch.equal(model.loss(t, labels), want), (t.dtype, t.device, t.stride())
    far = tokens.long()
    far[0] += 1 << 32
    out = tokens.clone()
    out[0] = -1
    assert torch.equal(model.loss(far, labels), model.loss(out, labels))
    if T == SMALL.T:
        _, ref = model.step(tokens, labels)
        for t in (tokens.long(), strided):
            _, g = model.step(t, labels)
            assert all(torch.equal(g[k], ref[k]) for k in ref)


def test_wide_experts_score():
    """Experts beyond the width that moe_forward_few takes."""
    say("case: example, wide experts")
    s = X.ModelShape(T=64, d=64, layers=1, vocab=50, n_routed=2, inter=32832, top_k=1)
    model = X.Model(s, seed=1)
    tokens, labels = X.make_batch(s, 2, ignored=0.0)
    loss = model.loss(tokens[:3].contiguous(), labels[:3].contiguous())
    assert loss.shape == (3,) and bool(torch.isfinite(loss).all()) and bool((loss > 0).all())
    assert torch.equal(loss, model.loss(tokens, labels)[:3])


def test_training_without_a_limit_forms_no_norm(monkeypatch):
    say("case: example, training without a limit")
    calls = []
    whole = X.clip
    monkeypatch.setattr(X, "clip", lambda *a: calls.append(a) or whole(*a))
    X.train(SMALL, 2)
    assert not calls
    X.train(SMALL, 2, max_norm=1.0)
    assert len(calls) == 2
    with pytest.raises(moe.MoEError):
        X.train(SMALL, 1, max_norm=float("nan"))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_that_is_not_finite_is_left_out(bad, monkeypatch):
    """One bad gradient element in the first of two steps: the parameters are those of the
    second step alone (the optimiser has seen nothing before)."""
    say(f"case: example, a gradient with {bad}")
    step, seen = X.Model.step, []

    def one_bad(self, tokens, labels):
        loss, grads = step(self, tokens, labels)
        if not seen:
            grads["0.w_down"][1, 2, 3] = bad
        seen.append(1)
        return loss, grads

    lines = []
    monkeypatch.setattr(X.Model, "step", one_bad)
    model = X.train(SMALL, 2, max_norm=0.5, log=lines.append)
    assert len(seen) == 2 and len(lines) == 2 and "no step" in lines[0]
    assert all(bool(torch.isfinite(p).all()) for p in model.params.values())
    monkeypatch.setattr(X.Model, "step", step)
    ref = X.Model(SMALL)
    opt = torch.optim.Adam(list(ref.params.values()), lr=0.01, betas=(0.9, 0.99))
    _, grads = ref.step(*X.make_batch(SMALL, 101))
    X.clip(grads, 0.5)
    for name, q in ref.params.items():
        q.grad = grads[name]
    opt.step()
    assert all(torch.equal(model.params[k], ref.params[k]) for k in ref.params)
