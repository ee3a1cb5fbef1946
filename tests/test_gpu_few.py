"""moe_forward_few against the fp64 oracle: every dtype combination, 1 to 64
tokens, shared experts, group-limited routing; its routing fields; tokens and
weights that are not finite; repeats, streams, graphs.

Bounds, for the experts' part y - u of all tokens, normwise:
  bf16 and f32 weights  2e-5: three fp32 sums of up to 8192 random terms (an error of
      sqrt(8192) 2^-24 = 5e-6 each at most), h as a pair of bf16 values (2^-17 =
      7.6e-6 of it at most), SiLU and the gates through expf-like functions (a few
      2^-24); with 2^-23 |y| for the last addition and its rounding.
  e4m3 weights          both sides decide h's codes, from an h that agrees to about
      1e-5: a value falls on the other side of a rounding border (spacing 2^-3 of it
      at most) with a probability of 1.6e-4, and moves by that step: sqrt(1.6e-4)
      2^-3 = 1.6e-3; few values may hold two such steps at once, sqrt(2 / values) 2^-3.
A bf16 y adds its rounding, 2^-8 |y| per element."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from moe_workloads import CONFIGS, PARITY_CONFIGS, make_inputs, to_numpy_f32
from oracle import moe_oracle as O
from tests.parity import check_routing, check_selection_grouped, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
P = PARITY_CONFIGS


def _case(name, T, **kw):
    cfg = P[name] if name in P else CONFIGS[name]
    return cfg.replace(T=T, name=f"{name}_T{T}" + "".join(f"_{k}{v}" for k, v in kw.items()), **kw)


CASES = [_case("small_bf16", t) for t in (1, 2, 16, 17, 32, 33, 64)] + [
    _case("small_bf16_ns2", 7), _case("small_bf16_ns2", 64), _case("small_bf16_ns0", 5), _case("small_bf16_ns0", 40),
    _case("small_fp32", 1), _case("small_fp32", 3), _case("small_fp32", 64), _case("tiny_fp32", 20),
    _case("small_fp8", 1), _case("small_fp8", 13), _case("small_fp8", 64), _case("small_fp8_ns2", 40),
    _case("dense_k_eq_n", 50), _case("one_token", 1), _case("wide_router", 64), _case("wide_router", 3, w_dtype="e4m3"),
    _case("small_bf16", 30, n_groups=4, topk_groups=2), _case("small_fp8", 9, n_groups=8, topk_groups=3),
    # one expert, one column block; a width of an odd number of 64-column runs
    _case("small_bf16", 11, n_routed=1, top_k=1, n_shared=0, d=64, inter=64),
    _case("small_bf16", 19, d=448, inter=704, n_routed=67, top_k=7),
    _case("small_fp32", 21, d=160, inter=224, n_routed=13, top_k=5, n_shared=3),
    # either side of where a launch of its own selects; 64, 128, 256 and 512 experts to a selection
    _case("small_bf16", 8, n_routed=64), _case("small_bf16", 9, n_routed=65), _case("small_fp8", 8, n_routed=130),
    _case("small_fp8", 8, n_routed=300, top_k=9), _case("small_bf16", 8, n_routed=320, n_groups=64, topk_groups=5),
    # columns shared among blocks, as many as there are
    _case("small_fp32", 30, n_routed=64, inter=256), _case("small_fp8", 50, d=128, n_routed=100, top_k=8, n_shared=2),
    _case("small_bf16", 64, d=64, inter=2048, n_routed=90, top_k=8, n_shared=2),
    # 17 to 32 tokens of more than 64 runs of K
    _case("small_bf16", 20, d=4160, inter=64),
]


def _run(cfg, inp, w, lib=moe.moe_forward_few, **kw):
    shape = moe.LayerShape.from_config(cfg)
    u, E, b = (t.to(DEV).contiguous() for t in (inp.u, inp.centroids, inp.bias))
    routing = moe.alloc_routing(shape)
    y = lib(shape, u, E, b, w, routing=routing, **kw)
    torch.cuda.synchronize()
    return y, routing


def _oracle(cfg, inp, sel):
    un, En, bn = to_numpy_f32(inp.u), to_numpy_f32(inp.centroids), inp.bias.numpy()
    f = to_numpy_f32
    routed = lambda e: (f(inp.w_gate_up[e]), f(inp.w_down[e]))  # noqa: E731
    shared = [(f(inp.ws_gate_up[s]), f(inp.ws_down[s])) for s in range(cfg.n_shared)]
    return O.layer_forward(un, En, bn, cfg.top_k, routed, cfg.n_routed, shared, selection=sel, fp8=cfg.fp8)["y"]


def _check_y(cfg, y, ref, un):
    got, part = y.float().cpu().numpy().astype(np.float64), ref - un
    if cfg.fp8:
        values = cfg.T * (cfg.top_k + cfg.n_shared) * cfg.inter
        tol = 2e-5 + np.sqrt(max(1.6e-4, 2.0 / values)) / 8
    else:
        tol = 2e-5
    err = np.linalg.norm(got - ref)
    store = np.linalg.norm(ref) * (2.0 ** -8 if cfg.out_dtype == "bf16" else 2.0 ** -23)
    say(f"  {cfg.name}: |dy| {err:.2e}, of the experts' part {err / np.linalg.norm(part):.1e}, bound {tol:.1e} + {store:.1e}")
    assert err <= tol * np.linalg.norm(part) + store
    # no token's row hides in the others'
    rows = np.linalg.norm(got - ref, axis=1)
    each = 8 * tol * np.linalg.norm(part, axis=1) + np.linalg.norm(ref, axis=1) * (2.0 ** -8 if cfg.out_dtype == "bf16" else 2.0 ** -23)
    assert (rows <= each).all(), np.nonzero(rows > each)


@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_few_follows_the_oracle(cfg):
    say(f"case: moe_forward_few {cfg.name}")
    inp = make_inputs(cfg, 0)
    y, routing = _run(cfg, inp, moe.prepare_weights(cfg, inp))
    un, En, bn = to_numpy_f32(inp.u), to_numpy_f32(inp.centroids), inp.bias.numpy()
    if cfg.grouped:
        r = O.route(un.astype(np.float64), En, bn, cfg.top_k, None, cfg.n_groups, cfg.topk_groups)
        check_selection_grouped(r, routing["topk_idx"].cpu().numpy(), cfg.top_k, cfg.n_groups, cfg.topk_groups)
    else:
        check_routing(routing, un, En, bn, cfg.top_k, cfg.n_routed)
    g = O.group_by_expert(routing["topk_idx"].cpu().numpy(), cfg.n_routed)
    for k, name in (("counts", "expert_counts"), ("offsets", "expert_offsets"), ("perm_token", "perm_token"), ("pos", "pos")):
        assert np.array_equal(np.asarray(g[k]).reshape(-1), routing[name].cpu().numpy().reshape(-1)), name
    _check_y(cfg, y, _oracle(cfg, inp, routing["topk_idx"].cpu().numpy()), un)


@pytest.mark.parametrize("name,T", [("bf16_d2048", 1), ("bf16_d2048", 37), ("fp8_d2048", 5), ("bf16_d7168", 3), ("fp8_d7168", 2)])
def test_few_full_width(name, T):
    cfg = CONFIGS[name].replace(T=T, name=f"{name}_T{T}")
    say(f"case: moe_forward_few {cfg.name}, full width")
    inp = make_inputs(cfg, 0, weights_device=DEV)
    y, routing = _run(cfg, inp, moe.prepare_weights(cfg, inp))
    sel = routing["topk_idx"].cpu().numpy()
    check_routing(routing, to_numpy_f32(inp.u), to_numpy_f32(inp.centroids), inp.bias.numpy(), cfg.top_k, cfg.n_routed)
    _check_y(cfg, y, _oracle(cfg, inp, sel), to_numpy_f32(inp.u))
    del inp
    torch.cuda.empty_cache()


@pytest.mark.parametrize("name", ["small_bf16", "small_fp8", "small_fp32"])
def test_few_agrees_with_the_layer(name):
    """The same selection as moe_forward's, and y but for the roundings moe_forward
    makes between its kernels (bf16 H and Y: 1e-2 of rms(y), the layer's bound)."""
    cfg = _case(name, 48)
    say(f"case: moe_forward_few and moe_forward, {cfg.name}")
    inp = make_inputs(cfg, 3)
    w = moe.prepare_weights(cfg, inp)
    y, r = _run(cfg, inp, w)
    y2, r2 = _run(cfg, inp, w, lib=moe.moe_forward)
    assert torch.equal(r["topk_idx"], r2["topk_idx"]) and torch.equal(r["pos"], r2["pos"])
    assert torch.allclose(r["topk_gate"], r2["topk_gate"], rtol=1e-5, atol=0)
    bound = (4e-2 if cfg.fp8 else 1e-2) * y2.float().square().mean().sqrt().item() + 2.0 ** -8 * y2.float().abs()
    assert bool(((y.float() - y2.float()).abs() <= bound).all())


def test_few_tokens_alone():
    """A token's row alone and among 63 others: the same but for the order of its sums
    (2e-5 of the experts' part, as against the oracle)."""
    cfg = _case("small_bf16_ns2", 64)
    say("case: moe_forward_few, tokens alone and together")
    inp = make_inputs(cfg, 1)
    w = moe.prepare_weights(cfg, inp)
    y, r = _run(cfg, inp, w)
    u = inp.u.to(DEV)
    for t in (0, 15, 16, 40, 63):
        shape = moe.LayerShape.from_config(cfg, T=1)
        one = moe.moe_forward_few(shape, u[t:t + 1].contiguous(), inp.centroids.to(DEV), inp.bias.to(DEV), w)
        part = (y[t] - u[t].float()).norm()
        assert float((one[0] - y[t]).norm()) <= 4e-5 * float(part) + 2.0 ** -22 * float(y[t].norm())


@pytest.mark.parametrize("name", ["small_bf16", "small_fp32"])
def test_few_keeps_what_is_not_finite_apart(name):
    """A NaN token's row is NaN, with K distinct experts; NaN and infinite weights
    reach the tokens that use them and no others; every other row keeps its bits."""
    cfg = _case(name, 20)
    say(f"case: moe_forward_few, not finite, {cfg.name}")
    inp = make_inputs(cfg, 2)
    w = moe.prepare_weights(cfg, inp)
    y, r = _run(cfg, inp, w)
    inp.u = inp.u.clone()
    inp.u[7, 3] = float("nan")
    y1, r1 = _run(cfg, inp, w)
    idx = r1["topk_idx"].cpu().numpy()
    assert np.array_equal(np.sort(idx[7]), np.arange(cfg.top_k))   # all scores NaN: the lowest experts
    keep = torch.arange(20) != 7
    assert torch.equal(r1["topk_idx"][keep], r["topk_idx"][keep]) and bool(torch.isnan(y1[7]).all())
    # rows are placed behind those of lower experts' new row, and summed as before
    assert torch.equal(y1[keep], y[keep])
    inp.u[7, 3] = 0.0
    y, r = _run(cfg, inp, w)
    e = int(r["topk_idx"][0, 0])
    uses = (r["topk_idx"] == e).any(1).cpu()
    assert 0 < int(uses.sum()) < 20
    w.w_gate_up[e, 5] = float("inf")
    w.w_down[e, :, 9] = float("nan")
    y2, _ = _run(cfg, inp, w)
    assert torch.equal(y2.cpu()[~uses], y.cpu()[~uses]) and not bool(torch.isfinite(y2.cpu()[uses]).any())


def test_few_empty_batch():
    cfg = _case("small_bf16", 0)
    say("case: moe_forward_few, no tokens")
    shape = moe.LayerShape.from_config(cfg)
    inp = make_inputs(_case("small_bf16", 1), 0)
    w = moe.prepare_weights(cfg, inp)
    routing = moe.alloc_routing(shape)
    for t in routing.values():
        t.fill_(-7)
    y = moe.moe_forward_few(shape, inp.u[:0].to(DEV), inp.centroids.to(DEV), inp.bias.to(DEV), w, routing=routing)
    assert y.shape == (0, cfg.d)
    assert not routing["expert_counts"].any() and not routing["expert_offsets"].any()


@pytest.mark.parametrize("name,T", [("small_bf16", 3), ("small_fp8", 40)])
def test_few_repeats_streams_graph(name, T):
    """Bit-identical repeats: into a used workspace, on a side stream, and replayed
    from a captured graph with new inputs and eager work in between."""
    cfg = _case(name, T)
    say(f"case: moe_forward_few repeats, {cfg.name}")
    inp = make_inputs(cfg, 5)
    w = moe.prepare_weights(cfg, inp)
    shape = moe.LayerShape.from_config(cfg)
    E, b = inp.centroids.to(DEV), inp.bias.to(DEV)
    us = [inp.u.to(DEV), inp.u.to(DEV).flip(0).contiguous(), (0.5 * inp.u.to(DEV)).contiguous()]
    want = [moe.moe_forward_few(shape, u, E, b, w) for u in us]
    ws = torch.full((moe.few_workspace_size(shape),), 0xFF, dtype=torch.uint8, device=DEV)
    for u, y in zip(us, want):
        assert torch.equal(moe.moe_forward_few(shape, u, E, b, w, workspace=ws), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.moe_forward_few(shape, us[1], E, b, w, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want[1])
    u, y = us[0].clone(), torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_few(shape, u, E, b, w, y=y, workspace=ws)
    for k in (1, 2, 0, 1):
        u.copy_(us[k])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]), k
        assert torch.equal(moe.moe_forward_few(shape, us[2], E, b, w), want[2])


def test_few_calls_at_once():
    """Two calls on two streams, a workspace each, over and over: each as alone."""
    say("case: moe_forward_few, two calls at once")
    cases = [(_case("small_bf16_ns2", 40), 1), (_case("small_fp8", 7), 2)]
    runs = []
    for cfg, seed in cases:
        inp = make_inputs(cfg, seed)
        w, shape = moe.prepare_weights(cfg, inp), moe.LayerShape.from_config(cfg)
        args = (shape, inp.u.to(DEV), inp.centroids.to(DEV), inp.bias.to(DEV), w)
        runs.append((args, moe.moe_forward_few(*args), moe.alloc_few_workspace(shape), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for args, _, ws, stream in runs:
            with torch.cuda.stream(stream):
                got.append(moe.moe_forward_few(*args, workspace=ws))
    torch.cuda.synchronize()
    for k, y in enumerate(got):
        assert torch.equal(y, runs[k % 2][1]), k


def test_few_graphs_share_a_workspace():
    """Two captured calls of different shapes on one workspace, replayed in turn."""
    say("case: moe_forward_few, two graphs, one workspace")
    cases = [_case("small_bf16", 64), _case("small_bf16", 2)]
    inp = make_inputs(cases[0], 4)
    w = moe.prepare_weights(cases[0], inp)
    E, b = inp.centroids.to(DEV), inp.bias.to(DEV)
    shapes = [moe.LayerShape.from_config(c) for c in cases]
    ws = torch.zeros(max(moe.few_workspace_size(s) for s in shapes), dtype=torch.uint8, device=DEV)
    us = [inp.u.to(DEV), inp.u[5:7].to(DEV).contiguous()]
    want = [moe.moe_forward_few(s, u, E, b, w) for s, u in zip(shapes, us)]
    ys = [torch.empty_like(y) for y in want]
    graphs = []
    for s, u, y in zip(shapes, us, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.moe_forward_few(s, u, E, b, w, y=y, workspace=ws)
    for k in (0, 1, 1, 0, 1, 0):
        ys[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[k], want[k])


def test_few_routing_in_part():
    """Any of the routing's fields alone, y the same."""
    cfg = _case("small_bf16", 12)
    say("case: moe_forward_few, routing in part")
    inp = make_inputs(cfg, 7)
    w, shape = moe.prepare_weights(cfg, inp), moe.LayerShape.from_config(cfg)
    y, whole = _run(cfg, inp, w)
    u, E, b = (t.to(DEV) for t in (inp.u, inp.centroids, inp.bias))
    for name in whole:
        part = {name: torch.full_like(whole[name], -3)}
        assert torch.equal(moe.moe_forward_few(shape, u, E, b, w, routing=part), y)
        assert torch.equal(part[name], whole[name]), name


def test_few_writes_nothing_else():
    """The bytes around y, and a workspace's beyond its size, stay as they were."""
    cfg = _case("small_bf16", 10)
    say("case: moe_forward_few, bytes around")
    inp = make_inputs(cfg, 6)
    w, shape = moe.prepare_weights(cfg, inp), moe.LayerShape.from_config(cfg)
    n, need = cfg.T * cfg.d, moe.few_workspace_size(shape)
    buf = torch.full((n + 128,), 7.0, device=DEV)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    y = buf[64:64 + n].view(cfg.T, cfg.d)
    moe.moe_forward_few(shape, inp.u.to(DEV), inp.centroids.to(DEV), inp.bias.to(DEV), w, y=y, workspace=ws[:need])
    assert bool((buf[:64] == 7).all()) and bool((buf[-64:] == 7).all()) and bool((ws[need:] == 0xA5).all())


def test_few_refuses_on_the_gpu():
    cfg = _case("small_bf16", 4)
    inp = make_inputs(cfg, 0)
    w, shape = moe.prepare_weights(cfg, inp), moe.LayerShape.from_config(cfg)
    u, E, b = inp.u.to(DEV), inp.centroids.to(DEV), inp.bias.to(DEV)
    for kw in (dict(u=u[:3]), dict(u=u.float()), dict(centroids=E[:-1]), dict(bias=b.double()), dict(y=torch.empty(4, 8, device=DEV)),
               dict(weights=moe.ExpertWeights(w.w_gate_up[1:], w.w_down, w.ws_gate_up, w.ws_down)),
               dict(weights=moe.ExpertWeights(w.w_gate_up, w.w_down, w.ws_gate_up, w.w_down)),
               dict(routing={"topk_idx": torch.empty(4, 1, dtype=torch.int32, device=DEV)}),
               dict(routing={"expert_counts": torch.empty(cfg.n_routed, device=DEV)}),
               dict(u=torch.zeros(4, 2 * cfg.d, device=DEV).bfloat16()[:, ::2])):
        with pytest.raises(ValueError):
            moe.moe_forward_few(shape, **{**dict(u=u, centroids=E, bias=b, weights=w), **kw})
    with pytest.raises(moe.MoEError) as e:
        moe.moe_forward_few(shape, u, E, b, w, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.MOE_ERR_WORKSPACE
    with pytest.raises(moe.MoEError) as e:
        moe.moe_forward_few(moe.LayerShape.from_config(cfg, T=65), torch.cat([u] * 17)[:65].contiguous(), E, b, w)
    assert e.value.code == B.MOE_ERR_UNSUPPORTED
