"""moe_forward_few where numbers end: what is not finite, scores below fp32's range,
scores that are level, and a token's selection in batches of other sizes."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from moe_workloads import PARITY_CONFIGS, make_inputs, to_numpy_f32
from oracle import moe_oracle as O
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(name, T, seed, **kw):
    cfg = PARITY_CONFIGS[name].replace(T=T, **kw)
    return cfg, make_inputs(cfg, seed)


def _call(cfg, inp, w, lib=moe.moe_forward_few):
    shape = moe.LayerShape.from_config(cfg)
    routing = moe.alloc_routing(shape)
    y = lib(shape, inp.u.to(DEV), inp.centroids.to(DEV), inp.bias.to(DEV), w, routing=routing)
    torch.cuda.synchronize()
    return y.cpu(), routing["topk_idx"].cpu()


@pytest.mark.parametrize("where", ["scale", "code", "down scale", "shared scale", "token"])
def test_few_fp8_keeps_what_is_not_finite(where):
    """A NaN among 8-bit weights or scales, an infinite token: no row that uses it is
    finite anywhere (its 1x128 tiles of H or u read as NaN), every other row keeps its bits."""
    cfg, inp = _inputs("small_fp8", 20, 2)
    say(f"case: moe_forward_few, 8 bits, not finite, {where}")
    w = moe.prepare_weights(cfg, inp)
    y, idx = _call(cfg, inp, w)
    e = int(idx[0, 0])
    uses = (idx == e).any(1)
    assert bool(torch.isfinite(y).all()) and 0 < int(uses.sum()) < cfg.T
    cols = slice(None)
    if where == "scale":          # 128 rows of the gate
        w.s_gate_up[e, 0, 0] = float("nan")
    elif where == "code":         # one column of H
        w.w_gate_up[e, 5, 7] = 0x7f
    elif where == "down scale":   # 128 columns of y
        w.s_down[e, 0, 0] = float("nan")
        cols = slice(0, 128)
    elif where == "shared scale":
        w.ss_gate_up[0, 0, 0] = float("nan")
        uses[:] = True
    else:
        inp.u = inp.u.clone()
        inp.u[7, 3] = float("inf")
        uses[:] = False
        uses[7] = True
    y2, idx2 = _call(cfg, inp, w)
    assert torch.equal(y2[~uses], y[~uses]) and torch.equal(idx2[~uses], idx[~uses])
    assert not bool(torch.isfinite(y2[uses][:, cols]).any())
    if where == "down scale":
        assert torch.equal(y2[:, 128:], y[:, 128:])


@pytest.mark.parametrize("name,T", [("small_bf16", 20), ("small_fp32", 20), ("small_bf16_ns2", 50)])
def test_few_infinite_weights(name, T):
    """An infinite element of w_down makes an infinity of its column of y, of
    moe_forward's sign, for the rows that use it; nothing else changes."""
    cfg, inp = _inputs(name, T, 4)
    say(f"case: moe_forward_few, an infinite weight, {name}")
    w = moe.prepare_weights(cfg, inp)
    y, idx = _call(cfg, inp, w)
    e = int(idx[0, 0])
    uses = (idx == e).any(1)
    assert 0 < int(uses.sum()) < cfg.T
    w.w_down[e, 4, 9] = float("inf")
    w.w_down[e, 17, 2] = -float("inf")
    y2, _ = _call(cfg, inp, w)
    want, _ = _call(cfg, inp, w, lib=moe.moe_forward)
    for col in (4, 17):
        assert bool(torch.isinf(y2[uses, col]).all()) and torch.equal(y2[uses, col], want[uses, col])
        assert torch.equal(y2[~uses, col], y[~uses, col])
    rest = [c for c in range(cfg.d) if c not in (4, 17)]
    assert torch.equal(y2[:, rest], y[:, rest])


@pytest.mark.parametrize("dtype,kw", [("bf16", {}), ("f32", {}), ("bf16", dict(n_groups=8, topk_groups=3))])
def test_few_selection_in_any_batch(dtype, kw):
    """A token's experts and gates are the same bits in every batch, also where scores
    are level: centroids [p, q] and [q, p] have the same score for rows [v, v], and the
    order of its sum alone says which is larger."""
    say(f"case: moe_forward_few, selection in batches of other sizes, {dtype} {kw}")
    T, d, N, K = 64, 8192, 48, 5
    shape = moe.LayerShape(T, d, N, 0, 64, K, dtype, dtype, "f32", kw.get("n_groups", 1), kw.get("topk_groups", 1))
    g = torch.Generator().manual_seed(11)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    half = lambda *s: torch.randn(s, generator=g).to(dt)  # noqa: E731
    v, p, q = half(T, d // 2), 0.02 * half(N // 2, d // 2), 0.02 * half(N // 2, d // 2)
    u = torch.cat([v, v], 1).to(DEV).contiguous()
    E = torch.stack([torch.cat([p, q], 1), torch.cat([q, p], 1)], 1).view(N, d).to(DEV).contiguous()
    b = torch.zeros(N, device=DEV)
    w = moe.ExpertWeights((0.01 * half(N, 128, d)).to(DEV), (0.01 * half(N, d, 64)).to(DEV))

    def run(n, at):
        s = moe.LayerShape(n, d, N, 0, 64, K, dtype, dtype, "f32", shape.n_groups, shape.topk_groups)
        r = moe.alloc_routing(s)
        moe.moe_forward_few(s, u[at:at + n].contiguous(), E, b, w, routing=r)
        return r["topk_idx"], r["topk_gate"]

    idx, gate = run(T, 0)
    for n, at in ((1, 0), (1, 63), (2, 5), (4, 30), (5, 17), (8, 40), (9, 3), (17, 20), (33, 31)):
        i2, g2 = run(n, at)
        assert torch.equal(i2, idx[at:at + n]) and torch.equal(g2, gate[at:at + n]), (n, at)


def _tiny_scores(T, d, N, dtype):
    """Rows f_t times ones and centroids whose entries are all z_e / d: with powers of two for
    f_t and d every logit is exact in fp32, whatever its sum's order.  z_e from -84 to
    -91.5: at f = 1 fp32 holds some scores and not others, at f = 2 none, at 1/2 all.
    The bias alone decides who is chosen."""
    f = 2.0 ** (np.arange(T) % 4 - 2)
    u = torch.tensor(f, dtype=torch.float32)[:, None].expand(T, d)
    z = -84.0 - 0.5 * ((7 * np.arange(N) + 5 * (np.arange(N) // 16)) % 16)
    E = (torch.tensor(z, dtype=torch.float32) / d)[:, None].expand(N, d)
    b = torch.tensor(0.01 * ((5 * np.arange(N)) % 16), dtype=torch.float32) + 1e-4 * torch.arange(N)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    return u.to(dt).contiguous().to(DEV), E.to(dt).contiguous().to(DEV), b.to(DEV)


def _check_tiny_gates(u, E, b, idx, gate, K):
    """Gates to 1e-4: logf and the logits' differences leave a few units in the last place of
    88 (2^-18 each, 4e-6), and 2^-21 of a score below the normal range; expf and the
    quotient a few 2^-24."""
    r = O.route(to_numpy_f32(u.cpu()).astype(np.float64), to_numpy_f32(E.cpu()), b.cpu().numpy(), K)
    assert np.array_equal(np.sort(r["idx"], 1), np.sort(idx, 1))
    s = O.affinities(to_numpy_f32(u.cpu()), to_numpy_f32(E.cpu()))
    want = O.normalised_gates(s, idx)
    assert np.isfinite(gate).all() and np.abs(gate - want).max() <= 1e-4, np.abs(gate - want).max()
    assert (np.abs(gate - want) <= 1e-4 * want + 2e-8).all()


@pytest.mark.parametrize("T,N,K,dtype", [(4, 16, 6, "bf16"), (1, 16, 4, "f32"), (40, 300, 8, "bf16"), (64, 100, 3, "f32")])
def test_few_scores_below_fp32(T, N, K, dtype):
    """Tokens whose selected scores are all, or in part, below what fp32 holds: the gates are
    still the scores' shares, and y is finite."""
    say(f"case: moe_forward_few, tiny scores, {T} tokens, {N} experts, {dtype}")
    d = 256
    u, E, b = _tiny_scores(T, d, N, dtype)
    shape = moe.LayerShape(T, d, N, 0, 64, K, dtype, dtype)
    g = torch.Generator().manual_seed(5)
    w = moe.ExpertWeights((0.1 * torch.randn((N, 128, d), generator=g)).to(u.dtype).to(DEV),
                          (0.1 * torch.randn((N, d, 64), generator=g)).to(u.dtype).to(DEV))
    r = moe.alloc_routing(shape)
    y = moe.moe_forward_few(shape, u, E, b, w, routing=r)
    assert bool(torch.isfinite(y).all())
    _check_tiny_gates(u, E, b, r["topk_idx"].cpu().numpy(), r["topk_gate"].cpu().numpy().astype(np.float64), K)
