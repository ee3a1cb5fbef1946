"""The operators of a model's two ends and of serving, measured: the whole layer for a few tokens (``forward_few``), the
embedding lookup with the first block's norm and its gradient (``embed``), and the global norm and clipping of the
gradients (``clip``).  Plain forms in 32 bits (``own`` false) beside the framework's calls (``own`` true).

Cases are dicts: ``op`` names the operator; ``train`` adds the embedding's gradient.
"""

import math

import torch

own = False

EPS = 1e-6
MAX_NORM = 1.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}

D2048 = dict(d=2048, N=64, S=2, I=1408, K=6, groups=1, keep=1)
D7168 = dict(d=7168, N=256, S=1, I=2048, K=8, groups=1, keep=1)


def listed():
    return [
        # one new token of one request through the d = 2048 layer: latency
        dict(name="few_1_d2048", op="few", T=1, w="bf16", out="f32", **D2048),
        # one new token through the d = 7168 layer: nine experts' weights
        dict(name="few_1_d7168", op="few", T=1, w="bf16", out="f32", **D7168),
        # four drafted tokens of one request, 8-bit weights
        dict(name="few_4_fp8_d7168", op="few", T=4, w="e4m3", out="bf16", **D7168),
        # thirteen requests on a small 8-bit layer: several tokens to an expert
        dict(name="few_13_fp8_small", op="few", T=13, w="e4m3", out="bf16", d=512, N=16, S=1, I=384, K=4, groups=1, keep=1),
        # thirty-two requests, group-limited routing (8 groups, at most 4): most of the layer's weights
        dict(name="few_32_d7168_g8", op="few", T=32, w="bf16", out="bf16", **dict(D7168, groups=8, keep=4)),
        # one new token entering the model: its row and the first block's norm
        dict(name="embed_1_d7168", op="embed", T=1, d=7168, V=65536, table="bf16", x="bf16", norm=True, grad="f32",
             pad=0.0, train=False),
        # a small model's step, an odd width, fp32 throughout, scaled rows
        dict(name="embed_train_odd", op="embed", T=517, d=1992, V=10007, table="f32", x="f32", norm=False, grad="f32",
             pad=0.3, train=True),
        # a training batch of the d = 2048 layer in bf16
        dict(name="embed_train_d2048", op="embed", T=4096, d=2048, V=65536, table="bf16", x="bf16", norm=True, grad="bf16",
             pad=0.0, train=True),
        # the throughput batch of the d = 7168 layer, fp32 gradient
        dict(name="embed_train_d7168", op="embed", T=8192, d=7168, V=65536, table="bf16", x="bf16", norm=True, grad="f32",
             pad=0.1, train=True),
        # the gradients of the small example model: two blocks and its vocabulary
        dict(name="clip_model_small", op="clip", kind="model", layers=2, vocab=1000, d=256, N=16, S=1, I=128, above=True),
        # many small parameters of odd sizes, slices of one buffer, some in bf16
        dict(name="clip_ragged_211", op="clip", kind="ragged", n=211, most=300000, above=True),
        # one d = 2048 layer's gradients
        dict(name="clip_layer_d2048", op="clip", kind="model", layers=1, vocab=1000, d=2048, N=64, S=2, I=1408, above=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "embed", "clip"])
    if op == "few":
        w = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
        step = 128 if w == "e4m3" else 64
        T = _log(rng, 1, 64)
        d, I = step * _log(rng, 1, 4096 // step), step * _log(rng, 1, 2048 // step)
        N = _log(rng, 8, 256)
        if rng.random() < 0.3:
            N, groups, keep = max(16, N // 8 * 8), 8, rng.choice([2, 4])
            K = rng.randint(1, min(8, keep * (N // 8)))
        else:
            groups = keep = 1
            K = rng.randint(1, 8)
        while T * K * I * d > 64 * 2 ** 26:   # within the largest listed case
            I = max(step, I // 2 // step * step)
            T = max(1, T // 2)
        return dict(op=op, T=T, w=w, out=rng.choice(["f32", "bf16"]), d=d, N=N, S=rng.randint(0, 2), I=I, K=K,
                    groups=groups, keep=keep)
    if op == "embed":
        train = rng.random() < 0.7
        return dict(op=op, T=_log(rng, 1, 8192), d=8 * _log(rng, 8, 896), V=_log(rng, 256, 65536),
                    table=rng.choice(["f32", "bf16"]), x=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.5,
                    grad=rng.choice(["f32", "bf16"]), pad=rng.choice([0.0, 0.0, 0.2, 1.0]), train=train)
    above = rng.random() < 0.7
    if rng.random() < 0.5:
        return dict(op=op, kind="ragged", n=_log(rng, 1, 400), most=_log(rng, 10, 1000000), above=above)
    return dict(op=op, kind="model", layers=rng.randint(1, 4), vocab=_log(rng, 200, 20000), d=64 * _log(rng, 1, 16),
                N=_log(rng, 4, 32), S=rng.randint(0, 2), I=64 * _log(rng, 1, 8), above=above)


# ---------------------------------------------------------------- inputs


def _weights(g, w, *size):
    """One kind of weight matrices [n, rows, cols] as {"w": .., "s": ..} (s: a scale per 128x128 block of e4m3 codes)."""
    if w != "e4m3":
        return {"w": torch.empty(size, dtype=DTYPES[w], device="cuda").normal_(0.0, 0.006, generator=g)}
    t = torch.empty(size, dtype=torch.bfloat16, device="cuda").normal_(0.0, 120.0, generator=g).clamp_(-448.0, 448.0)
    n, rows, cols = size
    s = (0.8 + 0.4 * torch.rand((n, rows // 128, cols // 128), generator=g, device="cuda")) * (0.006 / 120.0)
    return {"w": t.to(torch.float8_e4m3fn).view(torch.uint8), "s": s}


def _prepare_few(case, g):
    T, d, N, S, I, w = (case[k] for k in ("T", "d", "N", "S", "I", "w"))
    xd = DTYPES["f32" if w == "f32" else "bf16"]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    st = {"u": randn(T, d).to(xd), "E": (0.02 * randn(N, d)).to(xd), "b": 0.01 * randn(N)}
    st.update(gu=_weights(g, w, N, 2 * I, d), dn=_weights(g, w, N, d, I))
    if S:
        st.update(sgu=_weights(g, w, S, 2 * I, d), sdn=_weights(g, w, S, d, I))
    return st


def _tokens(case, g):
    """Tokens as text has them (the r-th commonest as often as 1 / r), some of them padding (-1) at the end."""
    T, V = case["T"], case["V"]
    rank = torch.exp(math.log(V) * torch.rand(T, generator=g, device="cuda", dtype=torch.float64)).long().clamp(1, V) - 1
    tokens = ((rank * 7919 + 13) % V).to(torch.int32)
    pad = int(round(case["pad"] * T))
    if pad:
        tokens[T - pad:] = -1
    return tokens


def _clip_sizes(case):
    if case["kind"] == "model":
        d, N, S, I = (case[k] for k in ("d", "N", "S", "I"))
        layer = [(d,), (d,), (1, d), (N, d), (N, 2 * I, d), (N, d, I)] + ([(S, 2 * I, d), (S, d, I)] if S else [])
        return [(case["vocab"], d), (d,), (case["vocab"], d)] + layer * case["layers"]
    # sizes from the case alone: 1 .. most, as many small as large ones
    n, most = case["n"], case["most"]
    return [(max(1, int(round(most ** (((k * 61) % n) / max(1, n - 1))))),) for k in range(n)]


def _prepare_clip(case, g):
    sizes = _clip_sizes(case)
    total = sum(math.prod(s) for s in sizes)
    std = 7.0 / math.sqrt(total)
    randn = lambda s: std * torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if case["kind"] == "model":
        grads = [randn(s) for s in sizes]
        out = [torch.empty_like(t) for t in grads]
        whole = out
    else:   # slices of two flat buffers, one after the other: any alignment
        half = [sum(s[0] for s in sizes[k::2]) for k in (0, 1)]
        flat = [randn(half[0] + 1), randn(half[1] + 1).bfloat16()]
        whole = [torch.zeros_like(t) for t in flat]
        grads, out, at = [], [], [1, 1]
        for k, (n,) in enumerate(sizes):
            lo = at[k % 2]
            at[k % 2] += n
            grads.append(flat[k % 2][lo:lo + n])
            out.append(whole[k % 2][lo:lo + n])
    return {"grads": grads, "out": out, "whole": whole, "max_norm": MAX_NORM if case["above"] else 100.0}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "few":
        return dict(_prepare_few(case, g), case=case)
    if case["op"] == "clip":
        return dict(_prepare_clip(case, g), case=case)
    T, d, V = case["T"], case["d"], case["V"]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case, "tokens": _tokens(case, g), "w": 1.0 + 0.1 * randn(d),
          "table": (randn(V, d) / math.sqrt(d)).to(DTYPES[case["table"]])}
    if case["train"]:
        st["dx"] = randn(T, d) / T
    return st


# ---------------------------------------------------------------- plain forms


def _e4m3(v):
    """What 8 bits keep of fp32 rows: 1x128 tiles, scale amax / 448, codes E4M3 to nearest even."""
    t = v.view(v.shape[0], -1, 128)
    amax = t.abs().amax(-1, keepdim=True)
    none = amax == 0
    inv = torch.where(none, torch.zeros_like(amax), torch.full_like(amax, 448.0) / amax)
    scale = torch.where(none, torch.ones_like(amax), amax / 448.0)
    return ((t * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() * scale).view(v.shape)


def _select(st, case):
    """(experts [T, K], gates [T, K]); scores in 64 bits, ties to the lower expert."""
    s = torch.sigmoid(st["u"].double() @ st["E"].double().t())
    v = s + st["b"].double()
    G = case["groups"]
    if G > 1:
        per = case["N"] // G
        q = min(-(-case["K"] // case["keep"]), per)
        score = v.view(case["T"], G, per).sort(dim=-1, descending=True).values[:, :, :q].sum(-1)
        kept = score.sort(stable=True, dim=-1, descending=True).indices[:, :case["keep"]]
        mask = torch.ones_like(score, dtype=torch.bool).scatter_(1, kept, False)
        v = v.masked_fill(mask.repeat_interleave(per, dim=1), -math.inf)
    idx = v.sort(stable=True, dim=-1, descending=True).indices[:, :case["K"]]
    s = s.gather(1, idx)
    return idx, (s / s.sum(-1, keepdim=True)).float()


def _take(m, idx):
    """Matrices idx of one kind of weights in 32 bits."""
    w = m["w"][idx]
    if "s" not in m:
        return w.float()
    n, rows, cols = w.shape
    w = w.view(torch.float8_e4m3fn).float().view(n, rows // 128, 128, cols // 128, 128)
    return (w * m["s"][idx][:, :, None, :, None]).view(n, rows, cols)


def _experts(gu, dn, idx, x, fp8):
    """SwiGLU experts idx[a] on rows x[a]."""
    I = dn["w"].shape[2]
    y = torch.bmm(_take(gu, idx), (_e4m3(x) if fp8 else x).unsqueeze(-1)).squeeze(-1)
    g, u = y[:, :I], y[:, I:]
    h = g / (1.0 + torch.exp(-g)) * u
    return torch.bmm(_take(dn, idx), (_e4m3(h) if fp8 else h).unsqueeze(-1)).squeeze(-1)


def _plain_few(st):
    case, u = st["case"], st["u"].float()
    T, d, K, S, fp8 = case["T"], case["d"], case["K"], case["S"], case["w"] == "e4m3"
    idx, gate = _select(st, case)
    y = _experts(st["gu"], st["dn"], idx.flatten(), u.repeat_interleave(K, 0), fp8).view(T, K, d)
    out = u + (y * gate.unsqueeze(-1)).sum(1)
    if S:
        shared = torch.arange(S, device=u.device).repeat(T)
        out = out + _experts(st["sgu"], st["sdn"], shared, u.repeat_interleave(S, 0), fp8).view(T, S, d).sum(1)
    return {"y": out.to(DTYPES[case["out"]])}


def _scale(case):
    return math.sqrt(case["d"])


def _plain_embed(st):
    case, tokens = st["case"], st["tokens"].long()
    keep = (tokens >= 0)[:, None]
    at = tokens.clamp(min=0)
    x = torch.where(keep, st["table"][at].float() * _scale(case), torch.zeros((), device=at.device)).to(DTYPES[case["x"]])
    out = {"x": x}
    if case["norm"]:
        xf = x.float()
        out["n"] = (xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * st["w"]).to(torch.bfloat16)
    if case["train"]:
        dx = torch.where(keep, st["dx"] * _scale(case), torch.zeros((), device=at.device))
        out["dtable"] = torch.zeros((case["V"], case["d"]), device=at.device).index_add_(0, at, dx).to(DTYPES[case["grad"]])
    return out


def _plain_clip(st):
    norm = torch.stack([t.double().square().sum() for t in st["grads"]]).sum().sqrt()
    factor = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm)).float()
    for t, o in zip(st["grads"], st["out"]):
        o.copy_(t.float() * factor)
    return {"norm": norm.float().view(1), "out": st["whole"]}


# ---------------------------------------------------------------- the framework's calls


def _own_few(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    c = st["case"]
    shape = moe.LayerShape(c["T"], c["d"], c["N"], c["S"], c["I"], c["K"], "f32" if c["w"] == "f32" else "bf16", c["w"],
                           c["out"], c["groups"], c["keep"])
    gu, dn, none = st["gu"], st["dn"], {"w": None}
    sgu, sdn = st.get("sgu", none), st.get("sdn", none)
    weights = moe.ExpertWeights(gu["w"], dn["w"], sgu["w"], sdn["w"], gu.get("s"), dn.get("s"), sgu.get("s"), sdn.get("s"))
    return {"y": moe.moe_forward_few(shape, st["u"], st["E"], st["b"], weights)}


def _own_embed(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    c = st["case"]
    shape = moe.EmbedShape(c["T"], c["d"], c["V"], table_dtype=c["table"], x_dtype=c["x"], grad_dtype=c["grad"],
                           scale=_scale(c), eps=EPS)
    x, n = moe.moe_embed(shape, st["tokens"], st["table"], w_next=st["w"] if c["norm"] else None)
    out = {"x": x}
    if c["norm"]:
        out["n"] = n
    if c["train"]:
        out["dtable"] = moe.moe_embed_backward(shape, st["tokens"], st["dx"])
    return out


def _own_clip(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    grads = moe.TensorList(st["grads"])
    sumsq = moe.moe_grad_sumsq(grads)
    return {"norm": moe.moe_grad_clip(grads, sumsq, st["max_norm"], out=moe.TensorList(st["out"])), "out": st["whole"]}


def run(state):
    op = state["case"]["op"]
    if op == "few":
        return _own_few(state) if own else _plain_few(state)
    if op == "embed":
        return _own_embed(state) if own else _plain_embed(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "few":
        T, d, N, S, I, K = (case[k] for k in ("T", "d", "N", "S", "I", "K"))
        hit = N * (1.0 - (1.0 - K / N) ** T)   # experts that T tokens choose, on average
        each = 3 * I * d
        weights = (hit + S) * each * SIZE[case["w"]] * (1.0 + (4.0 / 128 ** 2 if case["w"] == "e4m3" else 0.0))
        xs = 4 if case["w"] == "f32" else 2
        return {"bytes": weights + N * d * xs + 4 * N + T * d * (xs + SIZE[case["out"]]),
                "flops": 2.0 * T * ((K + S) * each + N * d)}
    if case["op"] == "embed":
        T, d, V = case["T"], case["d"], case["V"]
        live = T - int(round(case["pad"] * T))
        # each row of the table that a token names, once: ranks as often as 1 / r
        rows = min(live, V, 1 + live / math.log(V) * (1 + math.log(V * math.log(V) / max(live, 1) + 1))) if live else 0
        b = 4 * T + rows * d * SIZE[case["table"]] + T * d * SIZE[case["x"]]
        if case["norm"]:
            b += T * d * 2 + 4 * d
        if case["train"]:
            b += 4 * live * d + V * d * SIZE[case["grad"]]
        return {"bytes": b, "flops": T * d * (1 + (5 if case["norm"] else 0) + (2 if case["train"] else 0))}
    sizes = [math.prod(s) for s in _clip_sizes(case)]
    each = [4 if case["kind"] == "model" or k % 2 == 0 else 2 for k in range(len(sizes))]
    return {"bytes": 2 * sum(n * e for n, e in zip(sizes, each)) + 4, "flops": 3 * sum(sizes)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _kept_64(v):
    """The values that 8 bits keep of a float64 row of whole 128-column tiles; the format's rule fixes 32 bits for the
    scale, its reciprocal and their product with the value."""
    t = v.float().reshape(-1, 128)
    top = t.abs().max(dim=1, keepdim=True).values
    live = top > 0
    safe = torch.where(live, top, torch.ones_like(top))
    codes = torch.where(live, t * (torch.tensor(448.0, device=t.device) / safe), torch.zeros_like(t))
    codes = torch.clamp(codes, -448.0, 448.0).to(torch.float8_e4m3fn).double()
    return (codes * torch.where(live, safe / 448.0, torch.ones_like(safe)).double()).reshape(v.shape)


def _matrix_64(m, e):
    if "s" not in m:
        return m["w"][e].double()
    w = m["w"][e].view(torch.float8_e4m3fn).double()
    return w * m["s"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_few(st, case):
    fp8, I = case["w"] == "e4m3", case["I"]
    keep8 = _kept_64 if fp8 else (lambda v: v)
    u, E, b = st["u"].double(), st["E"].double(), st["b"].double().cpu()
    score = (1.0 / (1.0 + torch.exp(-(E @ u.t())))).t().cpu()
    out = u.clone()
    chosen = {}   # expert: [(token, gate)]
    for t in range(case["T"]):
        s = score[t]
        key = (s + b).tolist()
        allowed = range(case["N"])
        if case["groups"] > 1:
            per = case["N"] // case["groups"]
            q = min(math.ceil(case["K"] / case["keep"]), per)
            rank = sorted(range(case["groups"]), key=lambda j: (-sum(sorted(key[j * per:(j + 1) * per])[::-1][:q]), j))
            allowed = [e for e in allowed if e // per in rank[:case["keep"]]]
        picked = sorted(allowed, key=lambda e: (-key[e], e))[:case["K"]]
        total = sum(float(s[e]) for e in picked)
        for e in picked:
            chosen.setdefault(("gu", "dn", e), []).append((t, float(s[e]) / total))
    for e in range(case["S"]):
        chosen[("sgu", "sdn", e)] = [(t, 1.0) for t in range(case["T"])]
    for (gu, dn, e), rows in chosen.items():
        at = torch.tensor([t for t, _ in rows], device=u.device)
        gates = torch.tensor([g for _, g in rows], device=u.device, dtype=torch.float64)
        z = keep8(u[at]) @ _matrix_64(st[gu], e).t()
        h = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
        out[at] += gates[:, None] * (keep8(h) @ _matrix_64(st[dn], e).t())
    return {"y": out}


def _exact_embed(st, case):
    tokens, f = st["tokens"].long(), _scale(case)
    live = torch.nonzero(tokens >= 0).flatten()
    x = torch.zeros((case["T"], case["d"]), dtype=torch.float64, device=tokens.device)
    x[live] = st["table"].index_select(0, tokens[live]).double() * f
    out = {"x": x}
    if case["norm"]:
        kept = x.to(DTYPES[case["x"]]).double()   # the norm reads the rows as they are stored
        out["n"] = kept / (kept.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt() * st["w"].double()
    if case["train"]:
        out["dtable"] = torch.zeros((case["V"], case["d"]), dtype=torch.float64, device=tokens.device)
        out["dtable"].index_put_((tokens[live],), st["dx"][live].double() * f, accumulate=True)
    return out


def _exact_clip(st, case):
    total = sum((t.double() ** 2).sum().item() for t in st["grads"])
    norm = math.sqrt(total)
    factor = st["max_norm"] / norm if norm > st["max_norm"] else 1.0
    parts = [t.double() * factor for t in st["grads"]]
    if case["kind"] == "ragged":
        first = torch.zeros(1, dtype=torch.float64, device="cuda")
        parts = [torch.cat([first] + parts[k::2]) for k in (0, 1)]
    return {"norm": torch.tensor([norm], dtype=torch.float64), "out": parts}


def exact(case, seed):
    st = prepare(case, seed)
    return {"few": _exact_few, "embed": _exact_embed, "clip": _exact_clip}[case["op"]](st, case)
