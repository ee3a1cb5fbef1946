"""The layer's router and its backward for tokens whose selected scores are, all or in
part, below what fp32 holds: gates are still the scores' shares (64-bit oracle)."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from moe_workloads import PARITY_CONFIGS, make_inputs
from tests.parity import say
from tests.test_gpu_backward import TOL, _compare, _dy, _train_step
from tests.test_gpu_few_limits import _check_tiny_gates, _tiny_scores

pytestmark = pytest.mark.gpu
DEV = "cuda"


# experts over blocks too; a block a tile of tokens; K split over blocks
@pytest.mark.parametrize("T,d,N,K,dtype", [(1, 256, 16, 4, "bf16"), (70, 256, 300, 8, "f32"), (4100, 256, 16, 6, "bf16"),
                                           (4099, 256, 300, 8, "f32"), (8192, 2048, 256, 8, "bf16")])
def test_router_scores_below_fp32(T, d, N, K, dtype):
    say(f"case: moe_route, tiny scores, {T} x {d}, {N} experts, {dtype}")
    u, E, b = _tiny_scores(T, d, N, dtype)
    shape = moe.LayerShape(T, d, N, 0, 64, K, dtype, dtype)
    r = moe.moe_route(shape, u, E, b)
    _check_tiny_gates(u, E, b, r["topk_idx"].cpu().numpy(), r["topk_gate"].cpu().numpy().astype(np.float64), K)


@pytest.mark.parametrize("lift", [0.0, 4.0])
def test_backward_scores_below_fp32(lift):
    """The training step's gradients at the bounds of the other shapes.  One column of u is
    16 and lifts every logit to -86 - e/2 (in part below fp32's scores) or lower, with
    `lift` to -150 - e/2 (all of them)."""
    cfg = PARITY_CONFIGS["small_bf16"]
    say(f"case: moe_backward, tiny scores, lift {lift}")
    inp = make_inputs(cfg, 0)
    u, E = inp.u.clone(), inp.centroids.clone()
    u[:, 0] = 16.0
    E[:, 0] = -(5.375 + lift) - torch.arange(cfg.n_routed) / 32
    inp.u, inp.centroids = u, E
    inp.bias = 0.01 * torch.arange(cfg.n_routed, dtype=torch.float32).flip(0)
    dy = _dy(cfg)
    y, du, dE, grads, _, w = _train_step(cfg, inp, dy)
    shape = moe.LayerShape.from_config(cfg)
    r = moe.alloc_routing(shape)
    y2 = moe.moe_forward(shape, u.to(DEV), E.to(DEV), inp.bias.to(DEV), w, routing=r)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and bool(torch.isfinite(y).all())
    errs, _ = _compare(cfg, inp, dy, du, dE, grads, r["topk_idx"].cpu().numpy())
    say("  worst block ||d||/||ref||: " + ", ".join(f"{k} {v:.2e}" for k, v in errs.items()))
    for k, v in errs.items():
        assert v <= TOL, (k, v)
