"""Cases of the MXFP4 operators: quantisation, the 4-bit product, and the gated feed-forward block's
forward and backward on 4-bit operands.

Formats (OCP Microscaling v1.0, MXFP4): a value is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives) times the power of two that its block of 32 consecutive values along the contraction shares,
    e = clamp(floor(log2(max |x|)) - 2, -127, 125),     code = round_to_nearest_even(x / 2^e), at most 6.
Codes of a [rows, K] operand are bytes [rows, ceil(K/32) * 16], the value of even k in the low half byte.
Scales are bytes e + 127 in tiles of 128 rows x 4 blocks, [ceil(rows/128)][ceil(K/128)][32][4][4], the byte
of row r, block j at [r/128][j/4][r%32][r%128/32][j%4].
"""
import math

import torch

own = False

BF16, F32 = 0, 1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's activations on the way into a 4-bit product
        {"name": "quantize token", "op": "quantize", "rows": 1, "cols": 5120, "type": "bf16", "both": False},
        # fp32 master weights with a ragged edge, both orientations
        {"name": "quantize f32 ragged", "op": "quantize", "rows": 1000, "cols": 2088, "type": "f32", "both": True},
        # a training batch's activations or gradients (s=2048 b=4 h=5120), both orientations
        {"name": "quantize batch", "op": "quantize", "rows": 8192, "cols": 5120, "type": "bf16", "both": True},
        # one token through a row-parallel weight: reads the weight once
        {"name": "product token", "op": "product", "m": 1, "n": 5120, "k": 20480, "bias": True, "out": "bf16"},
        # ragged in every dimension
        {"name": "product ragged", "op": "product", "m": 150, "n": 272, "k": 136, "bias": True, "out": "f32"},
        # a short prompt through a wide layer, fp32 partial sums
        {"name": "product prompt", "op": "product", "m": 517, "n": 4096, "k": 1024, "bias": False, "out": "f32"},
        # a training batch's column layer (s=2048 b=4 h=5120 ffn=20480)
        {"name": "product batch", "op": "product", "m": 8192, "n": 20480, "k": 5120, "bias": False, "out": "bf16"},
        # serving: four streams, one token each
        {"name": "forward tokens", "op": "forward", "m": 4, "h": 5120, "ffn": 20480, "p": 4, "bias": False, "save": False},
        # serving: a ragged prompt chunk
        {"name": "forward chunk", "op": "forward", "m": 333, "h": 4096, "ffn": 16384, "p": 8, "bias": True, "save": False},
        # training forward (s=2048 b=4), pre-activations saved
        {"name": "forward batch", "op": "forward", "m": 8192, "h": 5120, "ffn": 20480, "p": 4, "bias": False, "save": True},
        # training backward of a small block, ragged token count (s=499 b=4), with bias gradients
        {"name": "backward small", "op": "backward", "m": 1996, "h": 1024, "ffn": 4096, "p": 4, "bias": True},
        # training backward of a large block (s=1024 b=4)
        {"name": "backward batch", "op": "backward", "m": 4096, "h": 5120, "ffn": 20480, "p": 4, "bias": False},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "forward", "forward", "backward"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 8, 5120, 8), "type": rng.choice(["bf16", "f32"]),
                "both": rng.random() < 0.6}
    if op == "product":
        f32 = rng.random() < 0.3
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 20480, 8), "k": _log(rng, 32, 1024 if f32 else 5120, 8),
                "bias": rng.random() < 0.5, "out": "f32" if f32 else "bf16"}
    p = rng.choice([1, 2, 4, 8])
    most = 8192 if op == "forward" else 4096
    c = {"op": op, "m": _log(rng, 1, most), "h": _log(rng, 256, 5120, 8 * p), "ffn": _log(rng, 1024, 20480, 128 * p), "p": p,
         "bias": rng.random() < 0.4}
    if op == "forward":
        c["save"] = rng.random() < 0.5
    return c


def _packed(rows, k):
    """Bytes of a 4-bit operand, codes and scales."""
    return rows * k * 17 / 32


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 if c["type"] == "bf16" else 4) + n * 2 * (2 if c["both"] else 1), "flops": n * (2 if c["both"] else 1)}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": _packed(m, k) + _packed(n, k) + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    m, h, f = c["m"], c["h"], c["ffn"]
    if c["op"] == "forward":
        return {"bytes": 2 * m * h + _packed(2 * f, h) + _packed(h, f) + 2 * m * h + (4 * m * f if c["save"] else 0),
                "flops": 6 * m * h * f}
    return {"bytes": 4 * m * h + 4 * m * f + _packed(h, 2 * f) + _packed(f, h) + 2 * m * h + 6 * h * f, "flops": 12 * m * h * f}


# ------------------------------------------------------------------ the plain forms, in 32 bits
def _round4(x):
    """x [rows, K] rounded to MXFP4 along K: (element values, exponents, both [rows, blocks, 32 | 1])."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -k % 32)).view(rows, -1, 32)
    _, ex = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(x.abs().amax(-1, keepdim=True) > 0, (ex - 3).clamp(-127, 125), torch.full_like(ex, -127))
    v = torch.ldexp(x, -e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(v / step) * step).clamp(-6, 6), e


def _fake4(x):
    """The values that x [rows, K] stands for after rounding to MXFP4 along K."""
    q, e = _round4(x)
    return torch.ldexp(q, e).view(x.shape[0], -1)[:, : x.shape[1]]


def _pack4(x):
    """Codes and tiled scales of x [rows, K]."""
    q, e = _round4(x)
    rows, blocks = q.shape[0], q.shape[1]
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + torch.where(q < 0, 8, 0).to(torch.uint8)).view(rows, -1, 2)
    codes = code[:, :, 0] + code[:, :, 1] * 16
    s = torch.zeros(-rows % 128 + rows, -blocks % 4 + blocks, dtype=torch.uint8, device=x.device)
    s[:rows, :blocks] = (e.view(rows, blocks) + 127).to(torch.uint8)
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes.contiguous(), s


def _unpack4(codes, scales, k):
    """The fp32 values [rows, k] of codes and tiled scales."""
    rows = codes.shape[0]
    c = torch.stack((codes & 15, codes >> 4), -1).view(rows, -1, 32).to(torch.int32)
    m = (c & 7).float()
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, (m - 4) * 2))
    v = torch.where(c >= 8, -v, v)
    s = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:rows, : v.shape[1]].to(torch.int32) - 127
    return torch.ldexp(v, s[:, :, None]).view(rows, -1)[:, :k]


def _gate(h):
    """Gate and up halves [rows, ffn] of packed columns (256 b + j: gate feature 128 b + j, then up)."""
    v = h.view(h.shape[0], -1, 2, 128)
    return v[:, :, 0].reshape(h.shape[0], -1), v[:, :, 1].reshape(h.shape[0], -1)


def _join(g, u):
    return torch.stack((g.view(g.shape[0], -1, 128), u.view(u.shape[0], -1, 128)), 2).view(g.shape[0], -1)


def _shards(w, p):
    """[rows, cols] as column shards [p, rows, cols / p]."""
    return w.view(w.shape[0], p, -1).transpose(0, 1).contiguous()


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "quantize":
        # activations with a few large channels, as a trained block's have
        x = normal(c["rows"], c["cols"]) * torch.exp(normal(1, c["cols"]))
        s["x"] = x.to(torch.bfloat16) if c["type"] == "bf16" else x
        return s
    if c["op"] == "product":
        s["a"], s["as"] = _pack4(normal(c["m"], c["k"]))
        s["b"], s["bs"] = _pack4(normal(c["n"], c["k"]) * c["k"] ** -0.5)
        s["bias"] = normal(c["n"]).to(torch.bfloat16) if c["bias"] else None
        return s
    m, h, f = c["m"], c["h"], c["ffn"]
    s["x"] = normal(m, h).to(torch.bfloat16)
    if c["op"] == "forward":
        s["w"], s["ws"] = _pack4(normal(2 * f, h) * h**-0.5)
        s["b"], s["bs"] = _pack4(normal(h, f) * f**-0.5)
        s["bw"] = (normal(2 * f) * 0.1).to(torch.bfloat16) if c["bias"] else None
        s["b2"] = (normal(h) * 0.1).to(torch.bfloat16) if c["bias"] else None
        return s
    s["w"], s["ws"] = _pack4(normal(h, 2 * f) * h**-0.5)
    s["b"], s["bs"] = _pack4(normal(f, h) * f**-0.5)
    s["h"] = normal(m, 2 * f).to(torch.bfloat16)
    s["dz"] = normal(m, h).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    bf = torch.bfloat16
    if c["op"] == "quantize":
        along = _fake4(s["x"]).to(bf)
        return [along, _fake4(s["x"].float().t()).to(bf)] if c["both"] else [along]
    if c["op"] == "product":
        d = _unpack4(s["a"], s["as"], c["k"]) @ _unpack4(s["b"], s["bs"], c["k"]).t()
        d = d if s["bias"] is None else d + s["bias"].float()
        return d.to(bf) if c["out"] == "bf16" else d
    h, f = c["h"], c["ffn"]
    if c["op"] == "forward":
        pre = _fake4(s["x"]) @ _unpack4(s["w"], s["ws"], h).t()
        pre = pre if s["bw"] is None else pre + s["bw"].float()
        gate, up = _gate(pre)
        y = _fake4(gate / (1 + torch.exp(-gate)) * up)
        z = y @ _unpack4(s["b"], s["bs"], f).t()
        z = z if s["b2"] is None else z + s["b2"].float()
        return [z.to(bf), pre.to(bf)] if c["save"] else [z.to(bf)]
    gate, up = _gate(s["h"].float())
    dz, x = s["dz"].float(), s["x"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dy = _fake4(dz) @ _unpack4(s["b"], s["bs"], h).t()
    dh = _join(dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig)
    dx = _fake4(dh) @ _unpack4(s["w"], s["ws"], 2 * f).t()
    dht = _fake4(dh.t())
    dw = _fake4(x.t()) @ dht.t()
    db = _fake4((gate * sig * up).t()) @ _fake4(dz.t()).t()
    out = [dx.to(bf), _shards(dw, c["p"]).to(bf), db.to(bf)]
    return out + [dh.sum(0).to(bf), dz.sum(0).to(bf)] if c["bias"] else out


def _run_own(s):
    from megatron_tensor_mlp_gb300 import tpmlp as T

    c = s["case"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "quantize":
        rows, cols, dt = c["rows"], c["cols"], BF16 if c["type"] == "bf16" else F32
        q, qs = T.mxfp4_empty(rows, cols)
        t, ts = T.mxfp4_empty(cols, rows) if c["both"] else (None, None)
        T.tpmlp_mxfp4_quantize(s["x"], q, qs, t, ts, rows, cols, cols, 1, dt)
        out = [new(rows, cols)]
        T.tpmlp_mxfp4_dequantize(q, qs, out[0], rows, cols)
        if c["both"]:
            out.append(new(cols, rows))
            T.tpmlp_mxfp4_dequantize(t, ts, out[1], cols, rows)
        return out
    if c["op"] == "product":
        f32 = c["out"] == "f32"
        d = new(c["m"], c["n"], dtype=torch.float32 if f32 else torch.bfloat16)
        T.tpmlp_mxfp4_matmul(s["a"], s["as"], s["b"], s["bs"], s["bias"], d, c["m"], c["n"], c["k"], F32 if f32 else BF16)
        return d
    m, h, f, p = c["m"], c["h"], c["ffn"], c["p"]
    backward = c["op"] == "backward"
    if "work" not in s:  # a workspace that the program keeps
        s["work"] = new(T.tpmlp_mxfp4_swiglu_ws_bytes(m, 1, h, f, p, backward), dtype=torch.uint8)
    if not backward:
        z, pre = new(m, h), new(m, 2 * f) if c["save"] else None
        T.tpmlp_mxfp4_swiglu_mlp_fwd(s["x"], s["w"], s["ws"], s["bw"], s["b"], s["bs"], s["b2"], z, pre, s["work"], m, 1, h, f, p)
        return [z, pre] if c["save"] else [z]
    dx, dw, db = new(m, h), new(p, h, 2 * f // p), new(f, h)
    dbw, db2 = (new(2 * f), new(h)) if c["bias"] else (None, None)
    T.tpmlp_mxfp4_swiglu_mlp_bwd(s["x"], s["w"], s["ws"], s["b"], s["bs"], s["h"], s["dz"], dx, dw, db, dbw, db2, s["work"],
                                 m, 1, h, f, p, grad_dt=BF16)
    return [dx, dw, db, dbw, db2] if c["bias"] else [dx, dw, db]


# ------------------------------------------------------------------ the same in 64 bits, from the definition
def _nearest(x):
    """x [rows, K] in 64 bits -> the MXFP4 values it is rounded to along K, by a table of magnitudes."""
    rows, k = x.shape
    blocks = torch.zeros(rows, (k + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    blocks[:, :k] = x
    blocks = blocks.reshape(-1, 32)
    top = blocks.abs().max(dim=1).values
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    # log2 may come out just beside a whole number, on either side
    power = power - (torch.exp2(power) > top).double() + (torch.exp2(power + 1) <= top).double()
    scale = torch.exp2(torch.where(top > 0, power - 2, torch.full_like(power, -127)).clamp(-127, 125))[:, None]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    between = (table[1:] + table[:-1]) / 2
    size = (blocks / scale).abs()
    low, high = torch.bucketize(size, between), torch.bucketize(size, between, right=True)
    index = torch.where(low % 2 == 0, low, high)  # at a tie the two differ: the even code
    return (table[index] * torch.sign(blocks) * scale).reshape(rows, -1)[:, :k]


def _values(codes, scales, k):
    """The values of codes and tiled scales in 64 bits, by table and by explicit place."""
    signed = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=codes.device)
    rows = codes.shape[0]
    v = torch.empty(rows, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    v[:, 0::2] = signed[(codes % 16).long()]
    v[:, 1::2] = signed[(codes // 16).long()]
    r = torch.arange(rows, device=codes.device)[:, None]
    j = torch.arange(v.shape[1] // 32, device=codes.device)[None, :]
    at = ((r // 128 * scales.shape[1] + j // 4) * 32 + r % 32) * 16 + r % 128 // 32 * 4 + j % 4
    power = torch.exp2(scales.reshape(-1)[at].double() - 127)
    return (v.reshape(rows, -1, 32) * power[:, :, None]).reshape(rows, -1)[:, :k]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantize":
        x = s["x"].double()
        return [_nearest(x), _nearest(x.t())] if c["both"] else [_nearest(x)]
    if c["op"] == "product":
        d = torch.matmul(_values(s["a"], s["as"], c["k"]), _values(s["b"], s["bs"], c["k"]).t())
        return d if s["bias"] is None else d + s["bias"].double()
    m, h, f = c["m"], c["h"], c["ffn"]
    gate_at = torch.arange(f, device="cuda") // 128 * 256 + torch.arange(f, device="cuda") % 128
    if c["op"] == "forward":
        pre = torch.matmul(_nearest(s["x"].double()), _values(s["w"], s["ws"], h).t())
        if s["bw"] is not None:
            pre = pre + s["bw"].double()
        gate, up = pre[:, gate_at], pre[:, gate_at + 128]
        z = torch.matmul(_nearest(gate * torch.sigmoid(gate) * up), _values(s["b"], s["bs"], f).t())
        if s["b2"] is not None:
            z = z + s["b2"].double()
        return [z, pre] if c["save"] else [z]
    pre, dz = s["h"].double(), s["dz"].double()
    gate, up = pre[:, gate_at], pre[:, gate_at + 128]
    del pre
    dy = torch.matmul(_nearest(dz), _values(s["b"], s["bs"], h).t())
    sig = torch.sigmoid(gate)
    dh = torch.empty(m, 2 * f, dtype=torch.float64, device="cuda")
    dh[:, gate_at] = dy * up * (sig + gate * sig * (1 - sig))
    dh[:, gate_at + 128] = dy * gate * sig
    db = torch.matmul(_nearest((gate * sig * up).t()), _nearest(dz.t()).t())
    del gate, up, sig, dy
    dx = torch.matmul(_nearest(dh), _values(s["w"], s["ws"], 2 * f).t())
    dw = torch.matmul(_nearest(s["x"].double().t()), _nearest(dh.t()).t())
    out = [dx, torch.stack(torch.chunk(dw, c["p"], dim=1)), db]
    return out + [dh.sum(0), dz.sum(0)] if c["bias"] else out
