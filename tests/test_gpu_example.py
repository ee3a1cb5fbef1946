"""The example model: its gradients against the oracle, layer by layer, and a
short training run that learns its task."""

import numpy as np
import pytest
import torch

from mixture_experts_layer_deepseekmoe_amd import binding as moe
from mixture_experts_layer_deepseekmoe_amd import example as X
from oracle import around_oracle as A
from oracle import moe_oracle as O
from tests.parity import say

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def test_step_gradients_follow_the_oracle():
    """One block, every gradient against the fp64 oracle's chain on the
    operands the kernels read (bf16 weights and rows, 8-bit checkpoints, the
    GPU's expert selection).  Bound 2e-2 normwise: the layer's backward is within
    1e-2 of the oracle on the same operands (its own tests), the loss's G and the
    bf16 rows between the operators add a rounding of 2^-8 each at most.  The
    gradients that sum a checkpoint of computed rows (w_out, gate, w_final): the
    oracle's rows differ from the GPU's by up to 2^-8, so their E4M3 roundings (a
    step of up to 2^-3) differ by sqrt(2^-8 2^-3) = 2.2e-2 in the root mean square;
    bound 5e-2."""
    say("case: example, one step's gradients")
    s = X.ModelShape(T=96, d=128, layers=1, vocab=200, n_routed=8, inter=64, top_k=2)
    model = X.Model(s, seed=1)
    tokens, labels = X.make_batch(s, 5, ignored=0.2)
    loss, grads = model.step(tokens, labels)
    p = {k: _np(v) for k, v in model.params.items()}
    b = lambda k: _np(model.params[k].bfloat16())  # noqa: E731
    bf = lambda a: _np(torch.from_numpy(a).bfloat16())  # noqa: E731
    tok, lab = tokens.cpu().numpy(), labels.cpu().numpy()
    eps = 1e-6
    x = p["embed"][tok]
    n = bf(A.block_in(x, p["0.w_in"], eps))
    routing = moe.moe_route(s.layer(), torch.from_numpy(n).bfloat16().cuda(), model.params["0.centroids"].bfloat16(),
                            model.bias[0])
    sel = routing["topk_idx"].cpu().numpy()
    routed = lambda e: (b("0.w_gate_up")[e], b("0.w_down")[e])  # noqa: E731
    shared = [(b("0.ws_gate_up")[0], b("0.ws_down")[0])]
    bias = np.zeros(s.n_routed, np.float32)
    y = O.layer_forward(n, b("0.centroids"), bias, s.top_k, routed, s.n_routed, shared, selection=sel)["y"]
    xo, _ = A.block_out(x, y, n, p["0.w_out"], p["0.gate"], 0, eps, 1.0)
    h = bf(A.block_in(xo, p["w_final"], eps))
    ref_loss, _, _ = A.vocab_loss(h, b("w_vocab"), lab)
    valid = lab >= 0
    assert abs(float(loss) - ref_loss.sum() / valid.sum()) <= 1e-2 * abs(float(loss))
    ref = {}
    dh, ref["w_vocab"], _ = A.vocab_loss_backward(h, b("w_vocab"), lab, valid / valid.sum())
    ck = lambda v: A.checkpoint(v.astype(np.float32))[2]  # noqa: E731
    dx, ref["w_final"], _, _ = A.block_in_backward(dh, None, None, ck(xo), p["w_final"], A.rstd(xo, eps), 1.0)
    z = y - n
    dy, ref["0.w_out"], ref["0.gate"], *_ = A.block_out_backward(dx, ck(z), p["0.w_out"], p["0.gate"], 0, A.rstd(z, eps))
    r = O.layer_backward(n, b("0.centroids"), bias, s.top_k, routed, s.n_routed, shared, dy.astype(np.float32),
                         selection=sel)
    dx, ref["0.w_in"], _, _ = A.block_in_backward(r["du"], dy, dx, ck(x), p["0.w_in"], A.rstd(x, eps), 1.0)
    ref["embed"] = np.zeros_like(p["embed"])
    np.add.at(ref["embed"], tok, dx)
    ref["0.ws_down"] = np.stack(r["dWs_down"])
    for name, want in ref.items():
        got = _np(grads[name])
        err = np.linalg.norm(got - want) / np.linalg.norm(want)
        say(f"  {name}: {err:.1e}")
        bound = 5e-2 if name in ("0.w_out", "0.gate", "w_final") else 2e-2
        assert got.shape == want.shape and err <= bound, (name, err)


def test_training_learns_the_task():
    """From log V at the start to below a quarter of it, and the right next
    token scores above another, one token at a time."""
    say("case: example, 60 training steps")
    s = X.ModelShape()
    losses = []
    model = X.train(s, 60, log=lambda m: losses.append(float(m.split()[-1])))
    say(f"  losses {losses}")
    assert losses[0] > 0.8 * np.log(s.vocab) and losses[-1] < 0.25 * np.log(s.vocab)
    t = torch.arange(0, s.vocab, 37, dtype=torch.int32, device="cuda")
    right = torch.cat([model.loss(q[None], (3 * q[None] + 7) % s.vocab) for q in t])
    wrong = torch.cat([model.loss(q[None], (3 * q[None] + 8) % s.vocab) for q in t])
    assert (right < wrong).float().mean() > 0.9
    # a token alone scores as it does in a batch, to the bf16 rounding of the rows between (2^-8 of
    # logits of order 10, twice)
    assert torch.allclose(right, model.loss(t, (3 * t + 7) % s.vocab), atol=0.1)
