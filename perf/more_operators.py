"""Cases of the mixture-of-experts operators and of layer normalisation: the norm ahead of a block, the routing
of tokens to experts, products grouped by expert with ragged sizes, and the combination of the experts' rows,
each with its backward.

Routing.  A token's k experts are those with its largest logits (a tie goes to the lower index; -inf is never
chosen, so a token of -inf alone is padding and has no rows).  Weights are the softmax over all experts or over
the chosen ones.  Rows are the chosen (token, slot) pairs sorted by expert, then token: expert e's are
offsets[e] .. offsets[e + 1] - 1, row r is of token row_token[r], slot j of token t has row slot_row[t, j]
(-1: not chosen).
Gated experts.  Columns of the first weight are packed in blocks of 256: 128 gate features, then the 128 up
features of the same indices; y = silu(gate) up.
"""
import math

import torch

own = False

BF16, F32 = 0, 1
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # serving: four streams' tokens on the way into a block
        {"name": "norm tokens", "op": "norm", "rows": 4, "h": 5120, "type": "bf16", "stats": False},
        # training in 32 bits, ragged rows of an odd width
        {"name": "norm backward odd", "op": "norm backward", "rows": 1996, "h": 1001, "type": "f32"},
        # a training batch (s=2048 b=4 h=5120)
        {"name": "norm backward batch", "op": "norm backward", "rows": 8192, "h": 5120, "type": "bf16"},
        # serving: four streams, one token each, many small experts
        {"name": "route tokens", "op": "route", "tokens": 4, "experts": 64, "k": 2, "type": "f32", "chosen": True, "backward": False},
        # a training batch (s=2048 b=4) with its backward, logits from a bf16 product
        {"name": "route batch", "op": "route", "tokens": 8192, "experts": 64, "k": 8, "type": "bf16", "chosen": False, "backward": True},
        # serving: the gated first layer for four tokens, which reads the weights of eight experts at most
        {"name": "experts tokens", "op": "gated", "tokens": 4, "experts": 64, "k": 2, "h": 1024, "ffn": 4096, "bias": False, "save": False},
        # serving: the second layer of a ragged prompt chunk
        {"name": "experts chunk", "op": "product", "tokens": 333, "experts": 8, "k": 2, "cols_in": 4096, "cols_out": 1024, "bias": True, "gather": False},
        # training forward of the gated first layer (s=2048 b=4 h=5120), pre-activations saved
        {"name": "experts batch", "op": "gated", "tokens": 8192, "experts": 8, "k": 2, "h": 5120, "ffn": 4096, "bias": False, "save": True},
        # training backward of small experts, ragged token count (s=499 b=4), with bias gradients
        {"name": "experts backward small", "op": "backward", "tokens": 1996, "experts": 16, "k": 2, "h": 1024, "ffn": 1024, "bias": True},
        # training backward of large experts (s=1024 b=4 h=5120)
        {"name": "experts backward batch", "op": "backward", "tokens": 4096, "experts": 8, "k": 2, "h": 5120, "ffn": 4096, "bias": False},
        # serving: one row of each of two experts for each of four tokens
        {"name": "combine tokens", "op": "combine", "tokens": 4, "k": 2, "h": 5120, "drop": False, "backward": False},
        # training batch, forward and backward; some slots have no row
        {"name": "combine batch", "op": "combine", "tokens": 8192, "k": 2, "h": 5120, "drop": True, "backward": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["norm", "norm backward", "route", "combine", "gated", "gated", "product", "product", "backward"])
    if op in ("norm", "norm backward"):
        c = {"op": op, "rows": _log(rng, 1, 8192), "h": _log(rng, 16, 5120, rng.choice([1, 8])), "type": rng.choice(["bf16", "bf16", "f32"])}
        return dict(c, stats=rng.random() < 0.5) if op == "norm" else c
    if op == "route":
        experts = _log(rng, 2, 256)
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts, "k": rng.randint(1, min(8, experts)),
                "type": rng.choice(["bf16", "f32"]), "chosen": rng.random() < 0.5, "backward": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "tokens": _log(rng, 1, 8192), "k": rng.randint(1, 4), "h": _log(rng, 64, 2560, 8), "drop": rng.random() < 0.5,
                "backward": rng.random() < 0.5}
    experts = rng.choice([4, 8, 16, 64])
    few = experts == 64  # many experts are small ones
    c = {"op": op, "tokens": _log(rng, 1, 8192 if op != "backward" else 4096), "experts": experts, "k": rng.choice([1, 2])}
    if op == "product":
        c.update(cols_in=_log(rng, 64, 1024 if few else 5120, 8), cols_out=_log(rng, 64, 1024 if few else 5120, 8), gather=rng.random() < 0.5)
    else:
        c.update(h=_log(rng, 128, 1024 if few else 5120, 8), ffn=_log(rng, 128, 1024 if few else 2048, 128))
    c["bias"] = rng.random() < 0.4
    if op == "gated":
        c["save"] = rng.random() < 0.5
    return c


def work(case):
    c = case
    if c["op"] in ("norm", "norm backward"):
        n, es = c["rows"] * c["h"], 2 if c["type"] == "bf16" else 4
        if c["op"] == "norm":
            return {"bytes": 2 * n * es + 2 * c["h"] * es + (8 * c["rows"] if c["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * es + 8 * c["rows"] + c["h"] * (es + 8), "flops": 14 * n}
    if c["op"] == "route":
        n, es = c["tokens"] * c["experts"], 2 if c["type"] == "bf16" else 4
        slots = c["tokens"] * c["k"]
        b = n * es + 16 * slots + 4 * c["experts"] + 4
        return {"bytes": b + (2 * n * es + 12 * slots if c["backward"] else 0), "flops": n * (c["k"] + 4)}
    if c["op"] == "combine":
        row, slots = 2 * c["h"], c["tokens"] * c["k"]
        b = (slots + c["tokens"]) * row + 8 * slots
        return {"bytes": b + (((2 * slots + c["tokens"]) * row + 12 * slots) if c["backward"] else 0),
                "flops": slots * c["h"] * (7 if c["backward"] else 2)}
    rows = c["tokens"] * c["k"]
    live = min(c["experts"], rows)  # experts with rows, at most
    if c["op"] == "product":
        a, b = c["cols_in"], c["cols_out"]
        return {"bytes": 2 * (c["tokens"] if c["gather"] else rows) * a + 2 * live * a * b + 2 * rows * b, "flops": 2 * rows * a * b}
    h, f = c["h"], c["ffn"]
    if c["op"] == "gated":
        return {"bytes": 2 * c["tokens"] * h + 4 * live * h * f + 2 * rows * f + (4 * rows * f if c["save"] else 0), "flops": 4 * rows * h * f}
    return {"bytes": 2 * c["tokens"] * h + 2 * rows * (2 * h + 3 * f) + 6 * live * h * f + 6 * c["experts"] * h * f, "flops": 12 * rows * h * f}


# ------------------------------------------------------------------ inputs
def _plan(ids, experts):
    """The rows of chosen experts ids [T, k] (-1: none): offsets, row_token, slot_row."""
    t, k = ids.shape
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(experts, device=ids.device)).sum(0)
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=ids.device), counts.cumsum(0)))
    place = torch.arange(t * k, device=ids.device)
    row_token = torch.where(place < offsets[-1], order // k, -1)
    slot_row = torch.empty_like(place)
    slot_row[order] = torch.where(place < offsets[-1], place, -1)
    return offsets.int(), row_token.int(), slot_row.view(t, k).int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    s = {"case": c}
    if c["op"] in ("norm", "norm backward"):
        rows, h, dt = c["rows"], c["h"], TYPES[c["type"]]
        # a residual stream: channels of different size and mean
        s["x"] = ((normal(rows, h) + 0.3 * normal(1, h)) * torch.exp(0.5 * normal(1, h)) + 0.2).to(dt)
        s["gamma"], s["beta"] = (1 + 0.2 * normal(h)).to(dt), (0.1 * normal(h)).to(dt)
        if c["op"] == "norm backward":  # what the forward saves
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt().float()
            s["dy"] = normal(rows, h).to(dt)
        return s
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["k"]
        x = (normal(t, e) + 0.5 * normal(1, e)).to(TYPES[c["type"]])
        some = torch.rand(t, generator=g, device="cuda")
        s["logits"] = x.masked_fill((some < 0.02)[:, None], -math.inf)  # padded tokens
        if c["backward"]:
            s["dw"] = normal(t, k)
        return s
    t, k = c["tokens"], c["k"]
    if c["op"] == "combine":
        ids = torch.rand(t, 8, generator=g, device="cuda").topk(k).indices
        s["rows"] = t * k
        if c["drop"]:  # one slot in twenty, as of padded tokens
            s["rows"] -= t * k // 20
            ids.view(-1)[torch.randperm(t * k, generator=g, device="cuda")[s["rows"]:]] = -1
        _, _, s["slot_row"] = _plan(ids, 8)
        s["o"] = normal(s["rows"], c["h"]).to(bf)
        s["w"] = torch.rand(t, k, generator=g, device="cuda")
        if c["backward"]:
            s["dz"] = normal(t, c["h"]).to(bf)
        return s
    # experts of different popularity
    e = c["experts"]
    ids = (normal(t, e) + 0.5 * normal(1, e)).topk(k).indices
    s["offsets"], s["row_token"], _ = _plan(ids, e)
    s["counts"] = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    rows = t * k
    if c["op"] == "product":
        a, b = c["cols_in"], c["cols_out"]
        s["x"] = normal(t if c["gather"] else rows, a).to(bf)
        s["w"] = (normal(e, a, b) * a**-0.5).to(bf)
        s["b"] = (0.1 * normal(e, b)).to(bf) if c["bias"] else None
        return s
    h, f = c["h"], c["ffn"]
    s["x"] = normal(t, h).to(bf)
    s["w1"] = (normal(e, h, 2 * f) * h**-0.5).to(bf)
    if c["op"] == "gated":
        s["b1"] = (0.1 * normal(e, 2 * f)).to(bf) if c["bias"] else None
        return s
    s["w2"] = (normal(e, f, h) * f**-0.5).to(bf)
    s["h"] = normal(rows, 2 * f).to(bf)
    gate, up = _halves(s["h"].float())
    s["y"] = (gate * torch.sigmoid(gate) * up).to(bf)
    s["do"] = normal(rows, h).to(bf)
    return s


def _halves(v):
    """Gate and up halves of packed columns."""
    v = v.view(v.shape[0], -1, 2, 128)
    return v[:, :, 0].reshape(v.shape[0], -1), v[:, :, 1].reshape(v.shape[0], -1)


def _packed(g, u):
    return torch.stack((g.view(g.shape[0], -1, 128), u.view(u.shape[0], -1, 128)), 2).view(g.shape[0], -1)


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _by_expert(x, counts, w, transposed=False):
    """Rows x, sorted by expert, times their experts' weights w [E, K, N] (or their transposes)."""
    parts = [p @ (w[e].float().t() if transposed else w[e].float()) for e, p in enumerate(torch.split(x, counts)) if counts[e]]
    return torch.cat(parts)


def _sums(x, counts):
    return torch.stack([p.sum(0) for p in torch.split(x, counts)])


def _weight_gradients(x, d, counts):
    return torch.stack([p.t() @ q for p, q in zip(torch.split(x, counts), torch.split(d, counts))])


def _run_plain(s):
    c = s["case"]
    bf = torch.bfloat16
    if c["op"] == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + 1e-5)
        y = ((x - mean) * rstd * s["gamma"].float() + s["beta"].float()).to(s["x"].dtype)
        return [y, mean[:, 0], rstd[:, 0]] if c["stats"] else [y]
    if c["op"] == "norm backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["gamma"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        return [dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)]
    if c["op"] == "route":
        x = s["logits"].float()
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        top, ids = top[:, : c["k"]], ids[:, : c["k"]]
        has = top > -math.inf
        size = torch.exp(x - torch.where(has[:, :1], top[:, :1], 0))
        total = torch.where(has, size.gather(1, ids), 0).sum(1) if c["chosen"] else size.sum(1)
        p = size / torch.where(total > 0, total, 1)[:, None]
        w = torch.where(has, p.gather(1, ids), 0)
        ids = torch.where(has, ids, -1)
        out = [ids.int(), w, *_plan(ids, c["experts"])]
        if c["backward"]:
            inner = (w * s["dw"]).sum(1, keepdim=True)
            dl = torch.zeros_like(x) if c["chosen"] else -p * inner
            back = w * (s["dw"] - inner) if c["chosen"] else w * s["dw"]
            out.append(dl.scatter_add_(1, ids.clamp(min=0).long(), torch.where(has, back, 0)).to(s["logits"].dtype))
        return out
    if c["op"] == "combine":
        at, there = s["slot_row"].clamp(min=0).long(), (s["slot_row"] >= 0)[:, :, None]
        rows = torch.where(there, s["o"][at].float(), 0)
        out = [(s["w"][:, :, None] * rows).sum(1).to(bf)]
        if c["backward"]:
            dz = s["dz"].float()[:, None]
            out.append(torch.empty_like(s["o"]))
            out[1][s["slot_row"][there[:, :, 0]].long()] = (s["w"][:, :, None] * dz).to(bf)[there[:, :, 0]]
            out.append((rows * dz).sum(2))
        return out
    counts = s["counts"]
    if c["op"] == "product":
        x = (s["x"][s["row_token"]] if c["gather"] else s["x"]).float()
        y = _by_expert(x, counts, s["w"])
        if s["b"] is not None:
            y = y + s["b"].float()[_expert_of(s)]
        return [y.to(bf)]
    x = s["x"][s["row_token"]].float()
    if c["op"] == "gated":
        pre = _by_expert(x, counts, s["w1"])
        if s["b1"] is not None:
            pre = pre + s["b1"].float()[_expert_of(s)]
        gate, up = _halves(pre)
        y = (gate / (1 + torch.exp(-gate)) * up).to(bf)
        return [y, pre.to(bf)] if c["save"] else [y]
    gate, up = _halves(s["h"].float())
    do = s["do"].float()
    dy = _by_expert(do, counts, s["w2"], True)
    sig = 1 / (1 + torch.exp(-gate))
    dh = _packed(dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig)
    out = [_by_expert(dh, counts, s["w1"], True).to(bf), _weight_gradients(x, dh, counts).to(bf),
           _weight_gradients(s["y"].float(), do, counts).to(bf)]
    return out + [_sums(dh, counts).to(bf), _sums(do, counts).to(bf)] if c["bias"] else out


def _expert_of(s):
    """The expert of every row."""
    place = torch.arange(s["row_token"].shape[0], dtype=torch.int32, device="cuda")
    return torch.searchsorted(s["offsets"][1:], place, right=True)


def _run_own(s):
    from megatron_tensor_mlp_gb300 import tpmlp as T

    c = s["case"]
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    new = lambda *shape, dtype=bf: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] in ("norm", "norm backward"):
        rows, h, dt = c["rows"], c["h"], BF16 if c["type"] == "bf16" else F32
        out = new(rows, h, dtype=s["x"].dtype)
        if c["op"] == "norm":
            mean, rstd = (new(rows, dtype=f32), new(rows, dtype=f32)) if c["stats"] else (None, None)
            T.tpmlp_layernorm_fwd(s["x"], s["gamma"], s["beta"], out, mean, rstd, rows, h, h, h, 1e-5, dt)
            return [out, mean, rstd] if c["stats"] else [out]
        if "work" not in s:  # a workspace that the program keeps
            s["work"] = new(T.tpmlp_layernorm_ws_bytes(rows, h), dtype=torch.uint8)
        dgamma, dbeta = new(h, dtype=f32), new(h, dtype=f32)
        T.tpmlp_layernorm_bwd(s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"], out, dgamma, dbeta, s["work"], rows, h, h, h, h, dt, F32)
        return [out, dgamma, dbeta]
    t, k = c["tokens"], c["k"]
    if c["op"] == "route":
        e, dt = c["experts"], BF16 if c["type"] == "bf16" else F32
        if "work" not in s:
            s["work"] = new(T.tpmlp_moe_route_ws_bytes(t, e, k), dtype=torch.uint8)
        ids, slot_row = new(t, k, dtype=i32), new(t, k, dtype=i32)
        w, offsets, row_token = new(t, k, dtype=f32), new(e + 1, dtype=i32), new(t * k, dtype=i32)
        T.tpmlp_moe_route(s["logits"], ids, w, offsets, row_token, slot_row, s["work"], t, e, k, int(c["chosen"]), dt)
        out = [ids, w, offsets, row_token, slot_row]
        if c["backward"]:
            out.append(torch.empty_like(s["logits"]))
            T.tpmlp_moe_route_bwd(s["logits"], ids, w, s["dw"], out[-1], t, e, k, int(c["chosen"]), dt)
        return out
    if c["op"] == "combine":
        h, rows = c["h"], s["rows"]
        out = [new(t, h)]
        T.tpmlp_moe_combine(s["o"], s["slot_row"], s["w"], out[0], t, rows, k, h)
        if c["backward"]:
            out += [new(rows, h), new(t, k, dtype=f32)]
            T.tpmlp_moe_combine_bwd(s["o"], s["slot_row"], s["w"], s["dz"], out[1], out[2], t, rows, k, h)
        return out
    e, rows, at = c["experts"], t * k, s["offsets"]
    if c["op"] == "product":
        a, b = c["cols_in"], c["cols_out"]
        y = new(rows, b)
        T.tpmlp_moe_matmul(s["x"], s["row_token"] if c["gather"] else None, at, s["w"], s["b"], y, None, t if c["gather"] else rows, rows, e, a, b)
        return [y]
    h, f = c["h"], c["ffn"]
    if c["op"] == "gated":
        y, pre = new(rows, f), new(rows, 2 * f) if c["save"] else None
        T.tpmlp_moe_matmul(s["x"], s["row_token"], at, s["w1"], s["b1"], y, pre, t, rows, e, h, 2 * f, act=T.ACT_SWIGLU)
        return [y, pre] if c["save"] else [y]
    dh, dx, dw1, dw2 = new(rows, 2 * f), new(rows, h), new(e, h, 2 * f), new(e, f, h)
    db1, db2 = (new(e, 2 * f), new(e, h)) if c["bias"] else (None, None)
    T.tpmlp_moe_matmul_dx(s["do"], at, s["w2"], s["h"], dh, rows, e, f, h, act=T.ACT_SWIGLU)
    T.tpmlp_moe_matmul_dx(dh, at, s["w1"], None, dx, rows, e, h, 2 * f)
    T.tpmlp_moe_matmul_dw(s["x"], s["row_token"], at, dh, dw1, db1, t, rows, e, h, 2 * f, grad_dt=BF16)
    T.tpmlp_moe_matmul_dw(s["y"], None, at, s["do"], dw2, db2, rows, rows, e, f, h, grad_dt=BF16)
    return [dx, dw1, dw2, db1, db2] if c["bias"] else [dx, dw1, dw2]


# ------------------------------------------------------------------ the same in 64 bits, from the definition
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        y = (x - mean) / torch.sqrt(var + 1e-5) * s["gamma"].double() + s["beta"].double()
        return [y, mean.squeeze(1), 1 / torch.sqrt(var + 1e-5).squeeze(1)] if c["stats"] else [y]
    if c["op"] == "norm backward":
        x, dy, gamma = s["x"].double(), s["dy"].double(), s["gamma"].double()
        mean, rstd = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1)
        h = c["h"]
        unit = (x - mean) * rstd
        a = (dy @ gamma).unsqueeze(1) / h
        b = torch.einsum("rh,rh,h->r", dy, unit, gamma).unsqueeze(1) / h
        return [(dy * gamma - a - unit * b) * rstd, torch.einsum("rh,rh->h", dy, unit), torch.einsum("rh->h", dy)]
    if c["op"] == "route":
        x, k = s["logits"].double(), c["k"]
        left, chosen = x.clone(), []
        for _ in range(k):  # the first of the largest ones left
            best = left.max(dim=1, keepdim=True).values
            at = (left == best).to(torch.uint8).argmax(dim=1, keepdim=True)
            chosen.append(torch.where(best > -math.inf, at, -1))
            left.scatter_(1, at, -math.inf)
        ids = torch.cat(chosen, 1)
        mask = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), (ids >= 0).double()) > 0
        inside = x.masked_fill(~mask, -math.inf) if c["chosen"] else x
        p = torch.softmax(inside, dim=1).nan_to_num(0)  # (a token of -inf alone has no softmax)
        w = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0)
        out = [None, w, None, None, None]
        if c["backward"]:
            d = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, s["dw"].double(), 0))
            out.append(p * (d - (p * d).sum(1, keepdim=True)))
        return out
    if c["op"] == "combine":
        t, k = c["tokens"], c["k"]
        place = torch.arange(t, device="cuda")[:, None].expand(t, k)[s["slot_row"] >= 0]
        row = s["slot_row"][s["slot_row"] >= 0].long()
        w = torch.zeros(s["rows"], dtype=torch.float64, device="cuda")
        w[row] = s["w"][s["slot_row"] >= 0].double()
        token = torch.empty_like(row)
        token[row] = place
        o = s["o"].double()
        out = [torch.zeros(t, c["h"], dtype=torch.float64, device="cuda").index_add_(0, token, o * w[:, None])]
        if c["backward"]:
            dz = s["dz"].double()
            dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
            dw[s["slot_row"] >= 0] = torch.einsum("rh,rh->r", o, dz[token])[row]
            out += [dz[token] * w[:, None], dw]
        return out
    ends = s["offsets"].tolist()
    span = [slice(a, b) for a, b in zip(ends[:-1], ends[1:])]
    rows = c["tokens"] * c["k"]
    if c["op"] in ("product", "gated"):
        x, w, b = s["x"].double(), s["w" if c["op"] == "product" else "w1"], s["b" if c["op"] == "product" else "b1"]
        if c["op"] == "gated" or c["gather"]:
            x = x.index_select(0, s["row_token"].long())
        y = torch.empty(rows, w.shape[2], dtype=torch.float64, device="cuda")
        for e, at in enumerate(span):
            torch.matmul(x[at], w[e].double(), out=y[at])
            if b is not None:
                y[at] += b[e].double()
        if c["op"] == "product":
            return [y]
        gate_at = torch.arange(c["ffn"], device="cuda") // 128 * 256 + torch.arange(c["ffn"], device="cuda") % 128
        out = torch.nn.functional.silu(y[:, gate_at]) * y[:, gate_at + 128]
        return [out, y] if c["save"] else [out]
    h, f = c["h"], c["ffn"]
    gate_at = torch.arange(f, device="cuda") // 128 * 256 + torch.arange(f, device="cuda") % 128
    pre, do, y = s["h"].double(), s["do"].double(), s["y"].double()
    x = s["x"].double().index_select(0, s["row_token"].long())
    gate, up = pre[:, gate_at], pre[:, gate_at + 128]
    sig = torch.sigmoid(gate)
    dx = torch.empty(rows, h, dtype=torch.float64, device="cuda")
    dh = torch.empty(rows, 2 * f, dtype=torch.float64, device="cuda")
    dw1 = torch.empty(c["experts"], h, 2 * f, dtype=torch.float64, device="cuda")
    dw2 = torch.empty(c["experts"], f, h, dtype=torch.float64, device="cuda")
    for e, at in enumerate(span):
        dy = torch.einsum("rh,fh->rf", do[at], s["w2"][e].double())
        part = torch.empty(dy.shape[0], 2 * f, dtype=torch.float64, device="cuda")
        part[:, gate_at] = dy * up[at] * (sig[at] + gate[at] * sig[at] * (1 - sig[at]))
        part[:, gate_at + 128] = dy * gate[at] * sig[at]
        dh[at] = part
        dx[at] = torch.einsum("rn,hn->rh", part, s["w1"][e].double())
        dw1[e] = torch.einsum("rh,rn->hn", x[at], part)
        dw2[e] = torch.einsum("rf,rh->fh", y[at], do[at])
    out = [dx, dw1, dw2]
    if c["bias"]:
        out += [torch.stack([dh[at].sum(0) for at in span]), torch.stack([do[at].sum(0) for at in span])]
    return out
