"""The bounds-checked build on the forward for a few tokens, the embedding and the
gradients' norm: every index check passes, and the results equal the release
build's bit for bit."""

import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from moe_workloads import PARITY_CONFIGS, make_inputs
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _both(fn):
    rel = fn()
    prev = B.use_library(B.DEBUG_LIB_PATH)
    try:
        dbg = fn()
    finally:
        B.restore_library(prev)
    assert len(rel) == len(dbg) and all(torch.equal(a, b) for a, b in zip(rel, dbg))


@pytest.mark.parametrize("name,T", [("small_bf16", 1), ("small_bf16_ns2", 64), ("small_fp32", 17), ("small_fp8", 13),
                                    ("wide_router", 40), ("small_fp8_ns2", 64), ("dense_k_eq_n", 33)])
def test_debug_build_few(name, T):
    say(f"case: debug build, moe_forward_few {name} T={T}")
    cfg = PARITY_CONFIGS[name].replace(T=T)
    inp = make_inputs(cfg, 0)
    w, shape = moe.prepare_weights(cfg, inp), moe.LayerShape.from_config(cfg)
    u, E, b = (t.to(DEV).contiguous() for t in (inp.u, inp.centroids, inp.bias))
    if T > 2:
        u[1] = float("nan")

    def run():
        routing = moe.alloc_routing(shape)
        y = moe.moe_forward_few(shape, u, E, b, w, routing=routing)
        return [torch.nan_to_num(y), *[routing[k] for k in ("topk_idx", "expert_counts", "expert_offsets", "perm_token", "pos")]]

    _both(run)


@pytest.mark.parametrize("T,d,V", [(1, 64, 10), (700, 1032, 300), (17000, 72, 70000)])
def test_debug_build_embed(T, d, V):
    say(f"case: debug build, embed {T} x {d}, {V} entries")
    g = torch.Generator().manual_seed(T)
    tok = (V ** torch.rand(T, generator=g)).int().to(DEV) - 1
    tok[::7] = -5
    table, dx, w = torch.randn((V, d), generator=g).to(DEV), torch.randn((T, d), generator=g).to(DEV), torch.ones(d, device=DEV)
    s = moe.EmbedShape(T, d, V)
    base = torch.ones((V, d), device=DEV)
    _both(lambda: [*moe.moe_embed(s, tok, table, w_next=w), moe.moe_embed_backward(s, tok, dx),
                   moe.moe_embed_backward(s, tok, dx, dtable=base.clone(), accumulate=True)])


def test_debug_build_grads():
    say("case: debug build, gradients")
    g = torch.Generator().manual_seed(1)
    gs = [torch.randn((k * k * 97 + 1,), generator=g).to(DEV) for k in range(120)]
    outs = [torch.empty(t.shape, dtype=torch.bfloat16, device=DEV) for t in gs]

    def run():
        s = moe.moe_grad_sumsq(gs)
        return [s, moe.moe_grad_clip(gs, s, 1.0, out=outs), *[o.clone() for o in outs]]

    _both(run)
