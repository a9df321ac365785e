"""Layer norm, routing, grouped products and the combination of rows in 64 bits, written from their definitions with
loops over rows, tokens and experts; and the bounds of the kernels' errors.

Bounds.  A product of K terms is added in fp32 in the tensor cores, 16 terms to an instruction; each addition may drop
what lies below the last place of the running sum (2^-23 of it), which is at most sum |x| |w|, so the sum is off by at
most (K / 16 + 16) 2^-23 sum |x| |w| (16 for the additions inside an instruction).  A result stored in bf16 is off by
2^-8 of itself more (half a step), and by half the smallest subnormal.
"""
import torch

U = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
TINY = 2.0**-133  # the smallest bf16 subnormal
D = torch.float64


def product_bound(k):
    return (k / 16 + 16) * 2.0**-23


def close(got, ref, extra, name=""):
    """|got - ref| within the rounding of got's type and extra, element by element; places of NaN and infinities alike."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    g = got.to(D)
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(g)), f"{name}: other places are not finite"
    if not isinstance(extra, torch.Tensor):
        extra = torch.full_like(ref, extra)
    limit = U[got.dtype] * ref.abs() + TINY + extra * (1 + U[got.dtype])
    over = torch.where(fine, (g - ref).abs() - limit, torch.zeros_like(ref))
    worst = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or float(over.max()) <= 0, (
        f"{name}: {int((over > 0).sum())} of {over.numel()} off, worst at {worst}: {float(g.flatten()[worst])} for "
        f"{float(ref.flatten()[worst])} (limit {float(limit.flatten()[worst])})")


# ------------------------------------------------------------------ layer norm
def norm(x, gamma, beta, eps):
    """(y, mean, rstd) of rows x, in 64 bits."""
    x = x.to(D)
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).sum(1) / x.shape[1] + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma.to(D)
    if beta is not None:
        y = y + beta.to(D)
    return y, mean, rstd


def norm_bwd(x, gamma, mean, rstd, dy):
    x, dy, mean, rstd = (t.to(D) for t in (x, dy, mean, rstd))
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma.to(D)
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    return rstd[:, None] * (g - a - xhat * b), (dy * xhat).sum(0), dy.sum(0)


# ------------------------------------------------------------------ routing
def route(logits, k, chosen):
    """(ids, weights, offsets, row_token, slot_row) of a CPU tensor, token by token."""
    x = logits.to(D)
    t, e = x.shape
    ids, weights = torch.full((t, k), -1, dtype=torch.int32), torch.zeros(t, k, dtype=D)
    for i in range(t):
        row = x[i].tolist()
        order = sorted(range(e), key=lambda j: (0 if row[j] != row[j] else 1, -row[j] if row[j] == row[j] else 0, j))
        best = [j for j in order[:k] if row[j] != float("-inf")]
        if not best:
            continue
        p = torch.softmax(x[i][best] if chosen else x[i], 0)
        for s, j in enumerate(best):
            ids[i, s] = j
            weights[i, s] = p[s] if chosen else p[j]
    rows = [(int(ids[i, s]), i, s) for i in range(t) for s in range(k) if ids[i, s] >= 0]
    rows.sort()
    offsets = torch.tensor([sum(r[0] < j for r in rows) for j in range(e + 1)], dtype=torch.int32)
    row_token, slot_row = torch.full((t * k,), -1, dtype=torch.int32), torch.full((t, k), -1, dtype=torch.int32)
    for r, (_, i, s) in enumerate(rows):
        row_token[r] = i
        slot_row[i, s] = r
    return ids, weights, offsets, row_token, slot_row


def route_bwd(logits, ids, dw, chosen):
    """dlogits by the chain rule through an explicit softmax Jacobian, token by token."""
    x = logits.to(D)
    out = torch.zeros_like(x)
    for i in range(x.shape[0]):
        best = [int(j) for j in ids[i] if j >= 0]
        if not best:
            continue
        at = best if chosen else list(range(x.shape[1]))
        p = torch.softmax(x[i][at], 0)
        jac = torch.diag(p) - p[:, None] * p[None, :]  # d p / d logits
        d = torch.zeros(len(at), dtype=D)
        for s, j in enumerate(best):
            d[at.index(j)] = dw[i, s].to(D)
        out[i, at] = jac @ d
    return out


# ------------------------------------------------------------------ products
def halves(v):
    v = v.reshape(v.shape[0], -1, 2, 128)
    return v[:, :, 0].reshape(v.shape[0], -1), v[:, :, 1].reshape(v.shape[0], -1)


def packed(g, u):
    return torch.stack((g.reshape(g.shape[0], -1, 128), u.reshape(u.shape[0], -1, 128)), 2).reshape(g.shape[0], -1)


def matmul(x, offsets, w, bias=None):
    """(rows of x times their experts' weights, the same of magnitudes); rows of no expert are NaN."""
    off = offsets.tolist()
    y = torch.full((x.shape[0], w.shape[2]), float("nan"), dtype=D, device=x.device)
    size = y.clone()
    for e in range(w.shape[0]):
        a, b = off[e], off[e + 1]
        if b > a:
            y[a:b] = x[a:b].to(D) @ w[e].to(D)
            size[a:b] = x[a:b].to(D).abs() @ w[e].to(D).abs()
            if bias is not None:
                y[a:b] += bias[e].to(D)
                size[a:b] += bias[e].to(D).abs()
    return y, size


def silu(g):
    return g * torch.sigmoid(g)


def dsilu(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


def dw(x, offsets, dy, experts):
    """(dW, the same of magnitudes, dbias, of magnitudes)"""
    off = offsets.tolist()
    x, dy = x.to(D), dy.to(D)
    part = [(x[a:b], dy[a:b]) for a, b in zip(off[:-1], off[1:])]
    assert len(part) == experts
    return (torch.stack([p.t() @ q for p, q in part]), torch.stack([p.abs().t() @ q.abs() for p, q in part]),
            torch.stack([q.sum(0) for _, q in part]), torch.stack([q.abs().sum(0) for _, q in part]))


# ------------------------------------------------------------------ combination
def combine(o, slot_row, weights):
    """(Z, the same of magnitudes), slot by slot."""
    t, k = slot_row.shape
    z = torch.zeros(t, o.shape[1], dtype=D, device=o.device)
    size = z.clone()
    for j in range(k):
        there = slot_row[:, j] >= 0
        at = slot_row[there, j].long()
        w = torch.ones(at.shape[0], dtype=D, device=o.device) if weights is None else weights[there, j].to(D)
        z[there] += w[:, None] * o[at].to(D)
        size[there] += (w[:, None] * o[at].to(D)).abs()
    return z, size
