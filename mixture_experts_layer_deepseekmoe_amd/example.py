"""A small language model of MoE blocks, trained and then scored token by token
with this package's operators only.

    python -m mixture_experts_layer_deepseekmoe_amd.example [--steps 60] [--max-norm 1]

Each block is norm -> MoE layer -> norm, gate and residual; the loss is the
cross entropy over the vocabulary.  The forward keeps 8-bit checkpoints of the
normed rows, so a block's x, y and its output are not kept for the backward.
The embedding brings the first block's norm; the gradients are clipped by their
common norm (--max-norm); up to 48 tokens at a time are scored by the layer's
forward for a few tokens.
The task: the next token is a fixed function of the current one.
"""

from __future__ import annotations

import argparse
import math
from dataclasses import dataclass
from typing import List

import torch

from . import binding as moe


@dataclass
class ModelShape:
    T: int = 512          # tokens of a batch
    d: int = 256
    layers: int = 2
    vocab: int = 1000
    n_routed: int = 16
    n_shared: int = 1
    inter: int = 128
    top_k: int = 4

    def layer(self, T=None) -> moe.LayerShape:
        return moe.LayerShape(self.T if T is None else T, self.d, self.n_routed, self.n_shared, self.inter, self.top_k)

    def block(self, T=None) -> moe.BlockShape:
        return moe.BlockShape(self.T if T is None else T, self.d, x_dtype="f32", n_dtype="bf16", y_dtype="f32")

    def embed(self, T=None) -> moe.EmbedShape:
        return moe.EmbedShape(self.T if T is None else T, self.d, self.vocab)

    def loss(self, T=None) -> moe.LossShape:
        return moe.LossShape(self.T if T is None else T, self.d, self.vocab)


# moe_forward_few is ahead or level up to here; its and moe_forward's time, bf16, us: d = 2048 48 tokens 257, 264, 56
# tokens 270, 264; d = 7168 48 tokens 2764, 2755, 64 tokens 3193, 3166; d = 256 64 tokens 32, 36.
FEW = 48


def layer_forward(s: ModelShape, T: int):
    """The layer's forward that scores T tokens: few ones by moe_forward_few, within its limit on the experts' width."""
    return moe.moe_forward_few if T <= FEW and s.inter <= 32768 else moe.moe_forward


class Model:
    """fp32 parameters (``params``); the products take bf16 copies."""

    def __init__(self, s: ModelShape, seed: int = 0):
        self.s = s
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda std, *sz: std * torch.randn(sz, generator=g, device="cuda")  # noqa: E731
        d, I, N, M = s.d, s.inter, s.n_routed, s.n_shared
        p = {"embed": rn(1.0, s.vocab, d), "w_final": torch.ones(d, device="cuda"), "w_vocab": rn(d ** -0.5, s.vocab, d)}
        for k in range(s.layers):
            p.update({f"{k}.w_in": torch.ones(d, device="cuda"), f"{k}.w_out": torch.ones(d, device="cuda"),
                      f"{k}.gate": torch.full((1, d), 0.5, device="cuda"), f"{k}.centroids": rn(d ** -0.5, N, d),
                      f"{k}.w_gate_up": rn(d ** -0.5, N, 2 * I, d), f"{k}.w_down": rn(I ** -0.5, N, d, I),
                      f"{k}.ws_gate_up": rn(d ** -0.5, M, 2 * I, d), f"{k}.ws_down": rn(I ** -0.5, M, d, I)})
        self.params = p
        self.bias = [torch.zeros(N, device="cuda") for _ in range(s.layers)]   # the router's, no gradient

    def _weights(self, k: int):
        b = lambda n: self.params[f"{k}.{n}"].bfloat16()  # noqa: E731
        return b("centroids"), moe.ExpertWeights(b("w_gate_up"), b("w_down"), b("ws_gate_up"), b("ws_down"))

    def _norm_after(self, k: int) -> torch.Tensor:
        return self.params[f"{k + 1}.w_in" if k + 1 < self.s.layers else "w_final"]

    def _tokens(self, tokens: torch.Tensor) -> torch.Tensor:
        """Tokens of any integer type, strides and device as moe_embed takes them (outside the vocabulary: a row of zeros)."""
        tokens = tokens.to(self.params["embed"].device)
        if tokens.dtype is not torch.int32:   # what int32 does not hold must not wrap into the vocabulary
            tokens = torch.where((tokens >= 0) & (tokens < self.s.vocab), tokens, -1).to(torch.int32)
        return tokens.contiguous()

    def forward(self, tokens: torch.Tensor, train: bool):
        """The final normed rows and, for training, what the backward needs."""
        s, p, T = self.s, self.params, tokens.numel()
        bs, ls, tokens = s.block(T), s.layer(T), self._tokens(tokens)
        keep: List[dict] = []
        new_save = lambda: moe.alloc_block_save(bs, e4m3=True) if train else None  # noqa: E731
        s_in = new_save()
        x, n = moe.moe_embed(s.embed(T), tokens, p["embed"], w_next=p["0.w_in"], save_next=s_in)
        for k in range(s.layers):
            cen, w = self._weights(k)
            if train:
                ws = moe.alloc_train_workspace(ls)
                y = moe.moe_forward_train(ls, n, cen, self.bias[k], w, ws)
            else:
                ws = None
                y = layer_forward(s, T)(ls, n, cen, self.bias[k], w)
            s_out, s_next = new_save(), new_save()
            x, n_next = moe.moe_block_out(bs, x, y, w=p[f"{k}.w_out"], gate=p[f"{k}.gate"], skip=n,
                                          w_next=self._norm_after(k), save=s_out, save_next=s_next)
            keep.append(dict(n=n, cen=cen, w=w, ws=ws, s_in=s_in, s_out=s_out))
            n, s_in = n_next, s_next
        return n, keep, s_in

    def loss(self, tokens: torch.Tensor, labels: torch.Tensor) -> torch.Tensor:
        """Each token's cross entropy (0 where the label is ignored)."""
        h, _, _ = self.forward(tokens, False)
        return moe.moe_vocab_loss(self.s.loss(tokens.numel()), h, self.params["w_vocab"].bfloat16(), labels)[0]

    def step(self, tokens: torch.Tensor, labels: torch.Tensor):
        """(mean loss over the labelled tokens, gradients by parameter name)."""
        s, p = self.s, self.params
        bs, ls, ss = s.block(), s.layer(), s.loss()
        h, keep, save = self.forward(tokens, True)
        w_vocab = p["w_vocab"].bfloat16()
        loss, lse = moe.moe_vocab_loss(ss, h, w_vocab, labels)
        valid = (labels >= 0) & (labels < s.vocab)
        count = valid.sum().clamp(min=1)
        grads = {}
        dh, grads["w_vocab"] = moe.moe_vocab_loss_backward(ss, h, w_vocab, labels, lse, valid.float() / count)
        dx, grads["w_final"] = moe.moe_block_in_backward(bs, dh, p["w_final"], save)
        for k in reversed(range(s.layers)):
            f = keep[k]
            dy, grads[f"{k}.w_out"], grads[f"{k}.gate"] = moe.moe_block_out_backward(
                bs, dx, f["s_out"], w=p[f"{k}.w_out"], gate=p[f"{k}.gate"])
            du, grads[f"{k}.centroids"], gw = moe.moe_backward(ls, f["n"], f["cen"], f["w"], dy, f["ws"])
            grads.update({f"{k}.w_gate_up": gw.dw_gate_up, f"{k}.w_down": gw.dw_down,
                          f"{k}.ws_gate_up": gw.dws_gate_up, f"{k}.ws_down": gw.dws_down})
            # n feeds the layer (du) and, negated, the skip (dy); x feeds the norm and the residual (dx)
            dx, grads[f"{k}.w_in"] = moe.moe_block_in_backward(bs, du, p[f"{k}.w_in"], f["s_in"], dn_sub=dy, do=dx)
        grads["embed"] = moe.moe_embed_backward(s.embed(), self._tokens(tokens), dx)
        return loss.sum() / count, grads


def clip(grads: dict, max_norm: float) -> torch.Tensor:
    """Scales all gradients, in place, by min(1, max_norm / norm); returns their norm."""
    tensors = moe.TensorList(grads.values())
    return moe.moe_grad_clip(tensors, moe.moe_grad_sumsq(tensors), max_norm)


def make_batch(s: ModelShape, seed: int, ignored: float = 0.1):
    """(tokens, labels): the label is 3 token + 7 modulo the vocabulary; some labels are ignored (-100)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, s.vocab, (s.T,), generator=g, device="cuda", dtype=torch.int32)
    labels = (3 * tokens + 7) % s.vocab
    labels[torch.rand(s.T, generator=g, device="cuda") < ignored] = -100
    return tokens, labels


def train(s: ModelShape, steps: int, lr: float = 0.01, log=lambda *a: None, max_norm: float = float("inf")) -> Model:
    """``max_norm``: the gradients are scaled down to this norm (all of them together) where theirs is larger; infinite:
    their norm is not formed.  A step whose norm is not finite is left out."""
    model = Model(s)
    opt = torch.optim.Adam(list(model.params.values()), lr=lr, betas=(0.9, 0.99))
    for k in range(steps):
        loss, grads = model.step(*make_batch(s, 100 + k))
        if max_norm != float("inf"):
            norm = clip(grads, max_norm).item()
            if not math.isfinite(norm):   # nothing was clipped: such gradients must not reach the parameters
                log(f"step {k}: no step, the gradients' norm is {norm}")
                continue
        for name, q in model.params.items():
            q.grad = grads[name]
        opt.step()
        if k % 10 == 0 or k + 1 == steps:
            log(f"step {k}: loss {loss.item():.4f}")
    return model


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--max-norm", type=float, default=float("inf"))
    args = ap.parse_args()
    s = ModelShape()
    model = train(s, args.steps, log=lambda *a: print(*a, flush=True), max_norm=args.max_norm)
    # scoring: one new token at a time
    for token in (1, 500, 999):
        t = torch.tensor([token], dtype=torch.int32, device="cuda")
        right = model.loss(t, (3 * t + 7) % s.vocab).item()
        wrong = model.loss(t, (3 * t + 8) % s.vocab).item()
        print(f"token {token}: log p(next) = {-right:.3f}, of another {-wrong:.3f}", flush=True)


if __name__ == "__main__":
    main()
