"""moe_embed and moe_embed_backward against the fp64 oracle: odd sizes, skewed
tokens, padding, checkpoints, accumulation, both sorts; repeats and graphs.

Bounds: x is one product, rounded once or twice (fp32 2^-24, a bf16 x 2^-8 more).  An
element of the gradient sums n fp32 terms in at most three levels of sums of at most
62 + n/32 terms, then one product and, with accumulate, one sum: with 2^-24 for each of
at most 62 + n/32 + 3 roundings of partial sums that the terms' sizes bound (n up to
8192: 321 2^-24 = 2e-5); a bf16 gradient 2^-8 of its value more."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_deepseekmoe_amd as moe
from mixture_experts_layer_deepseekmoe_amd import binding as B
from oracle import around_oracle as R
from oracle import ends_oracle as A
from tests.parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32, U16 = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tokens(kind, T, V, g):
    if kind == "one":        # a token of every row
        t = torch.full((T,), V // 2)
    elif kind == "few":      # three tokens, the last of the vocabulary among them
        t = torch.tensor([0, V // 3, V - 1])[torch.randint(0, 3, (T,), generator=g)]
    elif kind == "none":
        t = torch.where(torch.rand(T, generator=g) < 0.5, -1, V)
    elif kind == "distinct":
        t = torch.randperm(V, generator=g)[:T]
    else:                    # as text has them, some outside [0, V)
        t = (V ** torch.rand(T, generator=g)).long() - 1
        t[torch.rand(T, generator=g) < 0.1] = -100
        t[torch.rand(T, generator=g) < 0.05] = 2 ** 31 - 1
        t[torch.rand(T, generator=g) < 0.05] = V
    return t.to(torch.int32).to(DEV)


def _shape(T, d, V, **kw):
    return moe.EmbedShape(T, d, V, **kw)


@pytest.mark.parametrize("T,d,V,table,x", [(1, 64, 10, "f32", "f32"), (7, 256, 100, "bf16", "bf16"), (33, 1992, 50, "f32", "bf16"),
                                           (600, 8, 1000, "bf16", "f32"), (5, 7168, 300, "bf16", "bf16"), (513, 2056, 77, "f32", "f32"),
                                           (3, 32768, 5, "bf16", "f32")])
def test_embed_follows_the_oracle(T, d, V, table, x):
    say(f"case: embed {T} x {d}, {V} entries, {table} to {x}")
    g = torch.Generator().manual_seed(T + d)
    tok = _tokens("text", T, V, g)
    w = torch.randn((V, d), generator=g).to(DT[table]).to(DEV)
    wn = (1 + 0.1 * torch.randn(d, generator=g)).to(DEV)
    s = _shape(T, d, V, table_dtype=table, x_dtype=x, scale=1.7)
    got, none = moe.moe_embed(s, tok, w)
    assert none is None
    ref = A.embed(_np(w), tok.cpu().numpy(), float(np.float32(1.7)))
    bound = np.abs(ref) * (U32 + (U16 if x == "bf16" else 0)) * 1.01
    assert (np.abs(_np(got) - ref) <= bound).all()
    # the norm in the same pass: moe_block_in of x as stored, bit for bit
    bs = moe.BlockShape(T, d, x_dtype=x)
    save, save2 = moe.alloc_block_save(bs, e4m3=d % 128 == 0), moe.alloc_block_save(bs, e4m3=d % 128 == 0)
    got2, n = moe.moe_embed(s, tok, w, w_next=wn, save_next=save)
    assert torch.equal(got2, got) and torch.equal(n, moe.moe_block_in(bs, got, wn, save=save2))
    assert torch.equal(save.rstd, save2.rstd)
    if d % 128 == 0:
        assert torch.equal(save.codes, save2.codes) and torch.equal(save.scales, save2.scales)
    refn = R.block_in(_np(got), _np(wn), 1e-6)
    assert (np.abs(_np(n) - refn) <= np.abs(refn) * (U16 + 1e-5)).all()


def _backward(T, d, V, kind, grad="f32", accumulate=False, scale=0.3, seed=0):
    g = torch.Generator().manual_seed(seed + T + d + V)
    tok = _tokens(kind, T, V, g)
    dx = torch.randn((T, d), generator=g).to(DEV)
    outside = (tok < 0) | (tok >= V)
    dx[outside] = float("nan")   # rows of no token are not read
    base = torch.randn((V, d), generator=g).to(DT[grad]).to(DEV) if accumulate else None
    s = _shape(T, d, V, grad_dtype=grad, scale=scale)
    got = moe.moe_embed_backward(s, tok, dx, dtable=None if base is None else base.clone(), accumulate=accumulate)
    clean = torch.where(outside[:, None], torch.zeros((), device=DEV), dx)
    sc = float(np.float32(scale))
    b = None if base is None else _np(base)
    ref = A.embed_backward(_np(clean), tok.cpu().numpy(), V, sc, b)
    mag = A.embed_magnitude(_np(clean), tok.cpu().numpy(), V, sc, b)
    bound = (65 + T / 32) * U32 * mag + (U16 * np.abs(ref) * 1.01 if grad == "bf16" else 0)
    err = np.abs(_np(got) - ref)
    assert np.isfinite(_np(got)).all() and (err <= bound).all(), (err - bound).max()
    if accumulate:   # rows of no token keep their bits
        used = torch.zeros(V, dtype=torch.bool, device=DEV)
        used[tok[~outside].long()] = True
        assert torch.equal(got[~used], base[~used])
    return s, tok, dx, got


@pytest.mark.parametrize("kind", ["text", "one", "few", "none"])
@pytest.mark.parametrize("T,d,V,grad", [(1, 64, 10, "f32"), (31, 8, 7, "bf16"), (32, 264, 50, "f32"), (65, 1024, 300, "bf16"),
                                        (517, 1992, 1007, "f32"), (1000, 1032, 3, "f32"), (2100, 72, 4001, "bf16")])
def test_embed_backward_follows_the_oracle(T, d, V, grad, kind):
    say(f"case: embed backward {T} x {d}, {V} entries, {grad}, {kind}")
    _backward(T, d, V, kind, grad)


@pytest.mark.parametrize("kind", ["text", "one", "none"])
@pytest.mark.parametrize("T,d,V,grad", [(1, 64, 10, "f32"), (100, 1032, 40, "bf16"), (700, 128, 100000, "f32"),
                                        (9000, 8, 300, "f32"), (17000, 8, 300, "bf16")])
def test_embed_backward_accumulates(T, d, V, grad, kind):
    say(f"case: embed backward, added, {T} x {d}, {V} entries, {grad}, {kind}")
    _backward(T, d, V, kind, grad, accumulate=True)


@pytest.mark.parametrize("T,d,V,kind", [(16384, 8, 200, "text"), (16385, 8, 255, "text"), (16385, 8, 256, "few"), (20000, 16, 65535, "text"),
                                        (20001, 8, 65536, "distinct"), (40000, 8, 70000, "text"), (33000, 8, 1000, "one")])
def test_embed_backward_sorts_many_rows(T, d, V, kind):
    """Both sorts, on either side of their border, and keys of one, two and three digits."""
    say(f"case: embed backward, {T} rows sorted, {V} entries, {kind}")
    _backward(T, d, V, kind)


def test_embed_backward_far_rows():
    """A table whose rows lie beyond 2^31 elements: 2^24 entries of 136 columns, in bf16."""
    say("case: embed backward, 2^24 entries")
    T, d, V = 9, 136, 1 << 24
    tok = torch.tensor([0, V - 1, V - 1, 12345678, 7, V - 2, -1, V, 0], dtype=torch.int32, device=DEV)
    dx = torch.randn((T, d), generator=torch.Generator().manual_seed(1)).to(DEV)
    s = _shape(T, d, V, grad_dtype="bf16", table_dtype="bf16")
    g = moe.moe_embed_backward(s, tok, dx)
    used = [0, 7, 12345678, V - 2, V - 1]
    small = {v: i for i, v in enumerate(used)}
    ref = A.embed_backward(_np(dx), [small.get(int(v), -1) for v in tok], len(used), 1.0)
    assert (np.abs(_np(g[used]) - ref) <= 3 * U32 * 10 + 1.01 * U16 * np.abs(ref)).all()
    g[used] = 0
    assert not bool(g.any())
    table = g
    table[V - 1] = 3.0
    x, _ = moe.moe_embed(s, tok, table)
    assert bool((x[[1, 2]] == 3).all()) and not bool(x[[0, 3, 4, 5, 6, 7, 8]].any())


def test_embed_gradient_is_the_differences():
    """(f(table + h v) - f(table - h v)) / 2h of f = sum(x dx), linear: to the fp32
    roundings of x, 2^-24 (|table| + h |v|) |dx| summed over all terms, over h."""
    say("case: embed, differences")
    T, d, V = 50, 64, 20
    g = torch.Generator().manual_seed(3)
    tok = _tokens("text", T, V, g)
    table, v, dx = (torch.randn(n, generator=g).to(DEV) for n in ((V, d), (V, d), (T, d)))
    s = _shape(T, d, V, scale=0.7)
    h = 0.25
    f = lambda t: float((moe.moe_embed(s, tok, t)[0].double() * dx.double()).sum())  # noqa: E731
    num = (f(table + h * v) - f(table - h * v)) / (2 * h)
    ana = float((moe.moe_embed_backward(s, tok, dx).double() * v.double()).sum())
    size = float((moe.moe_embed(s, tok, table.abs() + h * v.abs())[0] * dx.abs()).sum())
    assert abs(num - ana) <= 4 * U32 * size / h


def test_embed_empty_batch():
    say("case: embed, no tokens")
    s = _shape(0, 64, 10)
    tok = torch.empty(0, dtype=torch.int32, device=DEV)
    x, n = moe.moe_embed(s, tok, torch.ones(10, 64, device=DEV), w_next=torch.ones(64, device=DEV))
    assert x.shape == (0, 64) and n.shape == (0, 64)
    g = torch.full((10, 64), 5.0, device=DEV)
    moe.moe_embed_backward(s, tok, torch.empty(0, 64, device=DEV), dtable=g, accumulate=True)
    assert bool((g == 5).all())
    moe.moe_embed_backward(s, tok, torch.empty(0, 64, device=DEV), dtable=g)
    assert not bool(g.any())


@pytest.mark.parametrize("T", [300, 17000])
def test_embed_repeats_streams_graph(T):
    say(f"case: embed repeats, {T} rows")
    d, V = 256, 500
    s, tok, dx, want = _backward(T, d, V, "text")
    want = want.clone()
    ws = torch.full((moe.embed_workspace_size(s),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(want, float("nan"))
    assert torch.equal(moe.moe_embed_backward(s, tok, dx, dtable=out, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.moe_embed_backward(s, tok, dx, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    tok2 = tok.flip(0).contiguous()
    want2 = moe.moe_embed_backward(s, tok2, dx).clone()
    want2_finite = torch.isfinite(want2)
    t, table = tok.clone(), torch.randn(V, d, device=DEV)
    x = torch.empty(T, d, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_embed(s, t, table, x=x)
        moe.moe_embed_backward(s, t, dx, dtable=out, workspace=ws)
    for tk, wt, ok in ((tok2, want2, want2_finite), (tok, want, None), (tok2, want2, want2_finite), (tok, want, None)):
        t.copy_(tk)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, moe.moe_embed(s, tk, table)[0])
        assert torch.equal(out, wt) if ok is None else torch.equal(out[ok], wt[ok])


def test_embed_writes_nothing_else():
    say("case: embed, bytes around")
    T, d, V = 70, 72, 33
    g = torch.Generator().manual_seed(9)
    tok = _tokens("text", T, V, g)
    s = _shape(T, d, V)
    need = moe.embed_workspace_size(s)
    buf = torch.full((V * d + 128,), 7.0, device=DEV)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    moe.moe_embed_backward(s, tok, torch.ones(T, d, device=DEV), dtable=buf[64:64 + V * d].view(V, d), workspace=ws[:need])
    assert bool((buf[:64] == 7).all()) and bool((buf[-64:] == 7).all()) and bool((ws[need:] == 0xA5).all())
    xb = torch.full((T * d + 128,), 7.0, device=DEV)
    moe.moe_embed(s, tok, torch.ones(V, d, device=DEV), x=xb[64:64 + T * d].view(T, d))
    assert bool((xb[:64] == 7).all()) and bool((xb[-64:] == 7).all())


def test_embed_refuses_on_the_gpu():
    s = _shape(4, 64, 10)
    tok, table = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(10, 64, device=DEV)
    for kw in (dict(tokens=tok.long()), dict(tokens=tok[:3]), dict(table=table[:9]), dict(table=table.bfloat16()),
               dict(w_next=torch.zeros(63, device=DEV)), dict(x=torch.zeros(4, 64, device=DEV).bfloat16())):
        with pytest.raises(ValueError):
            moe.moe_embed(s, **{**dict(tokens=tok, table=table), **kw})
    with pytest.raises(moe.MoEError) as e:
        moe.moe_embed(s, tok, table, n_next=torch.zeros(4, 64, device=DEV).bfloat16())
    assert e.value.code == B.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoEError) as e:
        moe.moe_embed_backward(s, tok, torch.zeros(4, 64, device=DEV), workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.MOE_ERR_WORKSPACE
