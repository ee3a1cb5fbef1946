"""The operators around the layer, measured: the norms before and after a block with its gate and residual scale
(``block_in``, ``block_out``), their 8-bit activation checkpoints, and the cross entropy over a vocabulary
(``vocab_loss``).  Plain forms in 32 bits (``own`` false) beside the framework's calls (``own`` true).

Cases are dicts: ``op`` names the operator, ``train`` adds its backward pass, ``ckpt`` lets the backward read the 8-bit
checkpoint instead of the rows themselves.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one new token of one request, entering a layer: pure latency
        dict(name="in_decode_1", op="block_in", T=1, d=2048, x="bf16", train=False, ckpt=False, chain=False),
        # a training batch of the d = 2048 layer, the residual stream in bf16, gradients chained through the layer's skip
        dict(name="in_train_d2048", op="block_in", T=4096, d=2048, x="bf16", train=True, ckpt=False, chain=True),
        # the throughput batch of the d = 7168 layer, its rows kept in 8 bits for the backward
        dict(name="in_ckpt_d7168", op="block_in", T=8192, d=7168, x="bf16", train=True, ckpt=True, chain=True),
        # one new token leaving a layer and entering the next: residual, then the next layer's norm
        dict(name="out_decode_1", op="block_out", T=1, d=7168, x="bf16", y="bf16", norm=True, gate_rows=0, skip=True,
             next=True, train=False, ckpt=False),
        # a serving batch of 256 single tokens (the decode batch of the d = 7168 layer)
        dict(name="out_decode_256", op="block_out", T=256, d=7168, x="bf16", y="f32", norm=True, gate_rows=0, skip=True,
             next=True, train=False, ckpt=False),
        # ragged requests of 129 tokens, each with a gate row of its own, an fp32 residual stream
        dict(name="out_train_odd", op="block_out", T=517, d=1992, x="f32", y="f32", norm=True, gate_rows=129, skip=False,
             next=False, train=True, ckpt=False),
        # the throughput batch of the d = 7168 layer, gated per channel, 8-bit checkpoint, with the next layer's norm
        dict(name="out_ckpt_d7168", op="block_out", T=8192, d=7168, x="bf16", y="f32", norm=True, gate_rows=0, skip=True,
             next=True, train=True, ckpt=True),
        # scoring one token: the vocabulary matrix is read once
        dict(name="loss_score_1", op="vocab_loss", T=1, d=2048, V=32000, masked=0.0, train=False),
        # scoring a short continuation over an odd vocabulary
        dict(name="loss_score_37", op="vocab_loss", T=37, d=7168, V=50001, masked=0.0, train=False),
        # a small model's step, most tokens masked (a prompt)
        dict(name="loss_train_small", op="vocab_loss", T=517, d=512, V=10007, masked=0.6, train=True),
        # a training batch of the d = 2048 layer
        dict(name="loss_train_d2048", op="vocab_loss", T=4096, d=2048, V=65536, masked=0.0, train=True),
        # the d = 7168 layer, a quarter of the tokens masked
        dict(name="loss_train_d7168", op="vocab_loss", T=4096, d=7168, V=65536, masked=0.25, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_in", "block_out", "vocab_loss", "vocab_loss"])
    train = rng.random() < 0.6
    if op == "vocab_loss":
        T, d, V = _log(rng, 1, 4096), 64 * _log(rng, 1, 112), _log(rng, 256, 65536)
        masked = rng.choice([0.0, 0.0, 0.1, 0.5, 0.9, 1.0])
        return dict(op=op, T=T, d=d, V=V, masked=masked, train=train)
    T, ckpt = _log(rng, 1, 8192), train and rng.random() < 0.5
    d = 128 * _log(rng, 1, 56) if ckpt else 8 * _log(rng, 8, 896)
    x = rng.choice(["bf16", "f32"])
    if op == "block_in":
        return dict(op=op, T=T, d=d, x=x, train=train, ckpt=ckpt, chain=rng.random() < 0.5)
    return dict(op=op, T=T, d=d, x=x, y=rng.choice(["bf16", "f32"]), norm=rng.random() < 0.8,
                gate_rows=rng.choice([0, 0, 1, _log(rng, 1, T)]), skip=rng.random() < 0.5, next=rng.random() < 0.5,
                train=train, ckpt=ckpt)


def _gate_count(case):
    return -(-case["T"] // case["gate_rows"]) if case["gate_rows"] else 1


def _rows(g, T, d, dtype, scale=1.0):
    """Rows as a residual stream has them: channels of unequal size, a few of them large."""
    ch = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    ch[:: max(1, d // 8)] *= 8.0
    return (torch.randn((T, d), generator=g, device="cuda") * ch * scale).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, d = case["T"], case["d"]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "vocab_loss":
        V = case["V"]
        w = (randn(V, d) * (1.5 / math.sqrt(d))).to(torch.bfloat16)
        labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        # the hidden rows lean toward their label, as a trained model's do
        h = (randn(T, d) + 3.0 * w[labels.long()].float()).to(torch.bfloat16)
        order = torch.argsort(torch.rand(T, generator=g, device="cuda"))
        masked = order[: int(round(case["masked"] * T))]
        labels[masked] = -100
        h[masked[::2]] = float("nan")   # what stands in a masked row must not matter
        st.update(h=h, w=w, labels=labels)
        if case["train"]:
            st.update(dloss=(0.5 + torch.rand(T, generator=g, device="cuda")) / T)
        return st
    st["w"] = 1.0 + 0.1 * randn(d)
    st["x"] = _rows(g, T, d, case["x"])
    if case["op"] == "block_in":
        if case["train"]:
            st.update(dn=randn(T, d))
            if case["chain"]:
                st.update(dn_sub=0.1 * randn(T, d), do=randn(T, d))
        return st
    st["y"] = _rows(g, T, d, case["y"], 0.5)
    if case["skip"]:
        st["skip"] = randn(T, d).to(torch.bfloat16)
    st["gate"] = 0.5 + 0.2 * randn(_gate_count(case), d)
    if case["next"]:
        st["w_next"] = 1.0 + 0.1 * randn(d)
    if case["train"]:
        st["do"] = randn(T, d)
    return st


# ---------------------------------------------------------------- plain forms


def _tiles(v):
    """(codes, scales) of 1x128 tiles: scale amax / 448, codes E4M3 to nearest even."""
    t = v.view(v.shape[0], -1, 128)
    amax = t.abs().amax(-1, keepdim=True)
    inv = torch.where(amax == 0, torch.zeros_like(amax), 448.0 / amax)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return (t * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(v.shape), scale.squeeze(-1)


def _untile(codes, scales):
    return (codes.float().view(codes.shape[0], -1, 128) * scales.unsqueeze(-1)).view(codes.shape)


def _plain_in(st):
    case, x, w = st["case"], st["x"].float(), st["w"]
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    out = {"n": (x * r * w).to(torch.bfloat16)}
    if not case["train"]:
        return out
    out["rstd"] = r.squeeze(-1)
    if case["ckpt"]:
        codes, scales = _tiles(x)
        out.update(codes=codes, scales=scales)
        x = _untile(codes, scales)
    dn = st["dn"] - st["dn_sub"] if case["chain"] else st["dn"]
    xh, a = x * r, dn * w
    dx = r * (a - xh * (a * xh).mean(-1, keepdim=True))
    out["dx"] = dx + st["do"] if case["chain"] else dx
    out["dw"] = (dn * xh).sum(0)
    return out


def _expand(gate, case):
    if not case["gate_rows"]:
        return gate
    return gate[torch.arange(case["T"], device=gate.device) // case["gate_rows"]]


def _plain_out(st):
    case, z = st["case"], st["y"].float()
    if case["skip"]:
        z = z - st["skip"].float()
    gate = _expand(st["gate"], case)
    r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) if case["norm"] else torch.ones_like(z[:, :1])
    w = st["w"] if case["norm"] else torch.ones_like(st["w"])
    xo = (st["x"].float() + gate * (z * r * w)).to(DTYPES[case["x"]])
    out = {"x_out": xo}
    if case["next"]:
        xf = xo.float()
        out["n_next"] = (xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * st["w_next"]).to(torch.bfloat16)
    if not case["train"]:
        return out
    if case["ckpt"]:
        codes, scales = _tiles(z)
        out.update(codes=codes, scales=scales)
        z = _untile(codes, scales)
    zh, do = z * r, st["do"]
    a = do * gate * w
    out["dy"] = r * (a - zh * (a * zh).mean(-1, keepdim=True)) if case["norm"] else a
    s = do * zh
    if case["norm"]:
        out["dw"] = (s * gate).sum(0)
    pad = _gate_count(case) * (case["gate_rows"] or case["T"]) - case["T"]
    s = torch.cat([s, s.new_zeros(pad, s.shape[1])]) if pad else s
    out["dgate"] = w * s.view(_gate_count(case), -1, s.shape[1]).sum(1)
    return out


def _plain_loss(st):
    h, w, lab = st["h"], st["w"].float(), st["labels"].long()
    valid = lab >= 0
    h = torch.where(valid[:, None], h, torch.zeros_like(h)).float()
    at = lab.clamp(min=0)[:, None]
    logits = h @ w.t()
    m = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - m)
    s = e.sum(-1, keepdim=True)
    lse = (m + torch.log(s)).squeeze(-1)
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(valid, lse - logits.gather(1, at).squeeze(1), zero), "lse": torch.where(valid, lse, zero)}
    if not st["case"]["train"]:
        return out
    dl = torch.where(valid, st["dloss"], zero)[:, None]
    G = e * (dl / s)
    G.scatter_add_(1, at, -dl)
    out["dh"] = (G @ w).to(torch.bfloat16)
    out["dw"] = (G.t() @ h).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the framework's calls


def _own_in(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    case = st["case"]
    shape = moe.BlockShape(case["T"], case["d"], x_dtype=case["x"], eps=EPS)
    if not case["train"]:
        return {"n": moe.moe_block_in(shape, st["x"], st["w"])}
    save = moe.alloc_block_save(shape, e4m3=case["ckpt"])
    n = moe.moe_block_in(shape, st["x"], st["w"], save=save)
    dx, dw = moe.moe_block_in_backward(shape, st["dn"], st["w"], save, x=None if case["ckpt"] else st["x"],
                                       dn_sub=st.get("dn_sub"), do=st.get("do"))
    out = {"n": n, "rstd": save.rstd, "dx": dx, "dw": dw}
    if case["ckpt"]:
        out.update(codes=save.codes.view(torch.float8_e4m3fn), scales=save.scales)
    return out


def _own_out(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    case = st["case"]
    shape = moe.BlockShape(case["T"], case["d"], x_dtype=case["x"], y_dtype=case["y"], gate_rows=case["gate_rows"],
                           eps=EPS)
    w = st["w"] if case["norm"] else None
    save = moe.alloc_block_save(shape, e4m3=case["ckpt"]) if case["train"] else None
    x_out, n_next = moe.moe_block_out(shape, st["x"], st["y"], w=w, gate=st["gate"], skip=st.get("skip"),
                                      w_next=st.get("w_next"), save=save)
    out = {"x_out": x_out}
    if case["next"]:
        out["n_next"] = n_next
    if not case["train"]:
        return out
    rows = {} if case["ckpt"] else {"y": st["y"], "skip": st.get("skip")}
    dy, dw, dgate = moe.moe_block_out_backward(shape, st["do"], save, w=w, gate=st["gate"], **rows)
    out.update(dy=dy, dgate=dgate)
    if case["norm"]:
        out["dw"] = dw
    if case["ckpt"]:
        out.update(codes=save.codes.view(torch.float8_e4m3fn), scales=save.scales)
    return out


def _own_loss(st):
    import mixture_experts_layer_deepseekmoe_amd as moe
    case = st["case"]
    shape = moe.LossShape(case["T"], case["d"], case["V"], dh_dtype="bf16", dw_dtype="bf16")
    loss, lse = moe.moe_vocab_loss(shape, st["h"], st["w"], st["labels"])
    out = {"loss": loss, "lse": lse}
    if case["train"]:
        out["dh"], out["dw"] = moe.moe_vocab_loss_backward(shape, st["h"], st["w"], st["labels"], lse, st["dloss"])
    return out


def run(state):
    op = state["case"]["op"]
    if op == "block_in":
        return _own_in(state) if own else _plain_in(state)
    if op == "block_out":
        return _own_out(state) if own else _plain_out(state)
    return _own_loss(state) if own else _plain_loss(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "vocab_loss":
        V, keep = case["V"], T - int(round(case["masked"] * case["T"]))
        b = 2 * d * (keep + V) + 4 * T + 8 * T
        f = 2.0 * keep * d * V
        if case["train"]:
            b += 2 * d * (T + V) + 4 * T
            f *= 3   # the logits, dh and dw; computing the logits again is not counted
        return {"bytes": b, "flops": f}
    n, row = T * d, T * d * (1 + 4 / 128)
    if case["op"] == "block_in":
        b = n * (SIZE[case["x"]] + 2) + 4 * d
        if case["train"]:
            b += n * (4 + 4) + 4 * T + 4 * d + (n * 8 if case["chain"] else 0) + (row if case["ckpt"] else 0)
        return {"bytes": b, "flops": n * (16 if case["train"] else 4)}
    b = n * (2 * SIZE[case["x"]] + SIZE[case["y"]] + (2 if case["skip"] else 0) + (2 if case["next"] else 0))
    b += 4 * d * (_gate_count(case) + 1 + case["next"])
    if case["train"]:
        b += n * (4 + 4) + 4 * T + 4 * d * (_gate_count(case) + 1) + (row if case["ckpt"] else 0)
    return {"bytes": b, "flops": n * (24 if case["train"] else 10)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _e4m3_64(v):
    """The values that 8 bits keep of float64 rows of whole 1x128 tiles.  The format's rule fixes 32 bits for the scale,
    its reciprocal and their product with the value."""
    t = v.float().reshape(v.shape[0], v.shape[1] // 128, 128)
    top = t.abs().max(dim=-1).values
    nothing = top == 0
    factor = (448.0 / top.masked_fill(nothing, 1.0)).masked_fill(nothing, 0.0)
    scale = (top / 448.0).masked_fill(nothing, 1.0)
    codes = torch.clamp(t * factor[..., None], min=-448.0, max=448.0).to(torch.float8_e4m3fn)
    return codes.reshape(v.shape), scale, (codes.double() * scale.double()[..., None]).reshape(v.shape)


def _norm_backward_64(g, w, v, r):
    """(dv, per-element weight gradient) of v r w with r = (mean v^2 + eps)^(-1/2), for the upstream g."""
    inner = (g * w * v).sum(dim=1, keepdim=True) / v.shape[1]
    return g * w * r - v * r ** 3 * inner, g * v * r


def _exact_in(st, case):
    x, w = st["x"].double(), st["w"].double()
    r = (x.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).pow(-0.5)
    out = {"n": x * w * r}
    if case["train"]:
        out["rstd"] = r[:, 0]
        if case["ckpt"]:
            out["codes"], out["scales"], x = _e4m3_64(x)
            out["codes"], out["scales"] = out["codes"].double(), out["scales"].double()
        g = st["dn"].double()
        if case["chain"]:
            g = g - st["dn_sub"].double()
        out["dx"], each = _norm_backward_64(g, w, x, r)
        if case["chain"]:
            out["dx"] = out["dx"] + st["do"].double()
        out["dw"] = each.sum(dim=0)
    return out


def _exact_out(st, case):
    x, z = st["x"].double(), st["y"].double()
    if case["skip"]:
        z = z - st["skip"].double()
    T, d, L = case["T"], case["d"], case["gate_rows"] or case["T"]
    which = torch.div(torch.arange(T, device=x.device), L, rounding_mode="floor")
    gate = st["gate"].double().index_select(0, which)
    if case["norm"]:
        w, r = st["w"].double(), (z.pow(2).sum(dim=1, keepdim=True) / d + EPS).pow(-0.5)
    else:
        w, r = x.new_ones(d), x.new_ones(T, 1)
    out = {"x_out": x + gate * w * z * r}
    if case["next"]:
        kept = out["x_out"].to(DTYPES[case["x"]]).double()   # the next norm reads the stream as it is stored
        out["n_next"] = kept * (kept.pow(2).sum(dim=1, keepdim=True) / d + EPS).pow(-0.5) * st["w_next"].double()
    if case["train"]:
        if case["ckpt"]:
            codes, scales, z = _e4m3_64(z)
            out["codes"], out["scales"] = codes.double(), scales.double()
        do = st["do"].double()
        if case["norm"]:
            out["dy"], each = _norm_backward_64(do * gate, w, z, r)
            out["dw"] = each.sum(dim=0)
        else:
            out["dy"] = do * gate
        out["dgate"] = x.new_zeros(_gate_count(case), d).index_add_(0, which, do * z * r * w)
    return out


def _exact_loss(st, case):
    T, V = case["T"], case["V"]
    lab = st["labels"].long()
    keep = torch.nonzero(lab >= 0).flatten()
    h, w, lab = st["h"][keep].double(), st["w"].double(), lab[keep]
    logits = torch.matmul(h, w.t())
    lse = torch.logsumexp(logits, dim=1)
    out = {"loss": h.new_zeros(T).index_copy_(0, keep, lse - logits[torch.arange(len(keep), device=h.device), lab]),
           "lse": h.new_zeros(T).index_copy_(0, keep, lse)}
    if case["train"]:
        G = torch.exp(logits.sub_(lse[:, None]))
        G[torch.arange(len(keep), device=h.device), lab] -= 1.0
        G *= st["dloss"].double()[keep][:, None]
        out["dh"] = h.new_zeros(T, case["d"]).index_copy_(0, keep, torch.matmul(G, w))
        out["dw"] = torch.matmul(G.t(), h) if len(keep) else h.new_zeros(V, case["d"])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"block_in": _exact_in, "block_out": _exact_out, "vocab_loss": _exact_loss}[case["op"]](st, case)
