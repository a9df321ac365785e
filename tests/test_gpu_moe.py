"""Routing, products grouped by expert and the combination of rows on the GPU, against 64 bits (tests/moe_ref.py)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import moe_ref as R  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN = float("nan")


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import tpmlp
    yield tpmlp
    tpmlp.tpmlp_device_status()


def rnd(*shape, seed=0, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=I32, device="cuda")


# ------------------------------------------------------------------ routing
def run_route(T, logits, k, chosen, dt):
    t, e = logits.shape
    new = lambda *s, dtype=I32: torch.full(s, 77, dtype=dtype, device="cuda")  # noqa: E731
    ids, w, off, rt, sr = new(t, k), new(t, k, dtype=F32), new(e + 1), new(t * k), new(t, k)
    ws = torch.full((max(T.tpmlp_moe_route_ws_bytes(t, e, k), 1),), 255, dtype=torch.uint8, device="cuda")
    T.tpmlp_moe_route(logits, ids, w, off, rt, sr, ws, t, e, k, chosen, dt)
    return ids, w, off, rt, sr


def weight_slack(w, logits, chosen):
    """expf is within 2 units in the last place, the difference it is of within half one of the largest logit's size; a sum
    of up to 1024 terms adds (5 + 32) half units; the quotient one."""
    x = torch.where(torch.isfinite(logits), logits, torch.zeros_like(logits)).to(R.D).abs().amax(1, keepdim=True)
    return w * 2.0**-24 * (2 * x + 48)


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 2), (4, 64, 8), (7, 5, 5), (31, 33, 3), (32, 8, 1), (33, 64, 4), (65, 128, 6),
                                   (300, 129, 8), (257, 257, 2), (130, 1024, 32), (515, 8, 2)])
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("chosen", [0, 1])
def test_route_and_backward(T, t, e, k, dt, chosen):
    logits = rnd(t, e, seed=t + e, scale=2.0, dtype=F32 if dt else BF)
    if t > 3:  # padding, ties, a token with fewer experts than slots
        logits[2] = -float("inf")
        logits[3] = 0.5
        logits[0, 1:] = -float("inf")
    ids, w, off, rt, sr = run_route(T, logits, k, chosen, dt)
    ref = R.route(logits.cpu(), k, chosen)
    assert torch.equal(ids.cpu(), ref[0])
    for got, want, name in ((off, ref[2], "offsets"), (rt, ref[3], "row_token"), (sr, ref[4], "slot_row")):
        assert torch.equal(got.cpu(), want), name
    R.close(w.cpu(), ref[1], weight_slack(ref[1], logits.cpu(), chosen), "weights")
    dw = rnd(t, k, seed=9, dtype=F32)
    dw = torch.where(ids >= 0, dw, NAN)  # not read where no expert was chosen
    dl = torch.full_like(logits, NAN)
    T.tpmlp_moe_route_bwd(logits, ids, w, dw, dl, t, e, k, chosen, dt)
    want = R.route_bwd(logits.cpu(), ref[0], dw.cpu(), chosen)
    # a product and two sums of up to k terms of weights that are themselves within weight_slack
    size = torch.nan_to_num(dw).abs().to(R.D).sum(1, keepdim=True).cpu()
    x = torch.nan_to_num(logits.cpu().float(), neginf=0).abs().amax(1, keepdim=True).to(R.D)
    R.close(dl.cpu(), want, size * 2.0**-24 * (4 * x + 128), "dlogits")


def test_route_orders_nan_and_infinities(T):
    inf = float("inf")
    x = torch.tensor([[0.0, NAN, 1.0, inf], [inf, 1.0, -inf, inf], [-inf, -0.0, 0.0, -inf], [-inf] * 4], device="cuda")
    ids, w, off, rt, sr = run_route(T, x, 3, 1, 1)
    assert ids.tolist() == [[1, 3, 2], [0, 3, 1], [1, 2, -1], [-1, -1, -1]]
    assert torch.isnan(w[0]).all() and torch.isnan(w[1]).any()
    assert w[2].tolist() == [0.5, 0.5, 0.0] and w[3].tolist() == [0.0, 0.0, 0.0]
    assert off.tolist() == [0, 1, 4, 6, 8]


def test_route_many_tokens_keeps_order(T):
    t, e, k = 100003, 16, 3
    logits = rnd(t, e, seed=3, dtype=F32)
    ids, w, off, rt, sr = run_route(T, logits, k, 1, 1)
    want = logits.topk(k, dim=1).indices.int()  # (no ties among these)
    assert torch.equal(ids, want)
    order = torch.sort(want.reshape(-1), stable=True).indices
    assert torch.equal(rt, (order // k).int())
    assert torch.equal(sr.reshape(-1)[order], torch.arange(t * k, dtype=I32, device="cuda"))
    assert torch.equal(off[1:], torch.bincount(want.reshape(-1), minlength=e).cumsum(0).int())


def test_route_of_no_tokens(T):
    off = torch.full((9,), 5, dtype=I32, device="cuda")
    T.tpmlp_moe_route(None, None, None, off, None, None, None, 0, 8, 2)
    assert off.tolist() == [0] * 9


# ------------------------------------------------------------------ products
COUNTS = [0, 1, 15, 16, 17, 0, 129, 255, 256, 257, 300, 513, 0]
# few rows an expert on average, which the forward takes on another kernel (tiles of 64 tokens, a split contraction)
FEW = [0, 1, 15, 16, 17, 0, 63, 64, 65, 130, 300] + [0] * 20
SHAPES = [(8, 8), (64, 256), (72, 136), (200, 520), (1032, 264)]


def case(counts, K, gather, seed=0, tokens=None, behind=37):
    """Rows by counts and some behind the last, offsets, and X with the tokens of the rows (or the rows themselves)."""
    off = offsets_of(counts)
    rows = sum(counts) + behind
    if not gather:
        return rows, off, None, rnd(rows, K, seed=seed)
    tokens = tokens or max(rows // 2, 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    src = torch.randint(0, tokens, (rows,), generator=g, device="cuda", dtype=I32)
    return rows, off, src, rnd(tokens, K, seed=seed)


@pytest.mark.parametrize("K,N", SHAPES + [(4104, 136)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("counts", [COUNTS, FEW, [3, 0, 70], [100, 20, 129, 64, 0]], ids=["many", "few", "three", "middle"])
def test_matmul(T, K, N, gather, out, counts):
    rows, off, src, x = case(counts, K, gather, seed=K)
    e = len(counts)
    w, b = rnd(e, K, N, seed=2, scale=K**-0.5), rnd(e, N, seed=3)
    for i in (i for i, c in enumerate(counts) if c == 0):
        w[i] = NAN  # experts without rows
    y = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, b, y, None, x.shape[0], rows, e, K, N, out_dt=0 if out == BF else 1)
    n = sum(counts)
    ref, size = R.matmul((x if src is None else x[src.long()])[:n], off, w, b)
    R.close(y[:n], ref, R.product_bound(K) * size, "Y")
    assert (y[n:] == 7.0).all()  # rows behind the last


@pytest.mark.parametrize("counts", [[300, 0, 70, 513, 2], [30, 0, 7, 51, 2, 129]])
def test_matmul_of_whole_numbers_is_exact(T, counts):
    """Sums that bf16 holds: every place of every tile, without a tolerance."""
    K, N = 80, 392
    rows, off, src, _ = case(counts, K, True, behind=0)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-1, 2, (rows // 2, K), generator=g, device="cuda").to(BF)
    w = torch.randint(-1, 2, (len(counts), K, N), generator=g, device="cuda").to(BF)
    y = torch.empty(rows, N, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, None, y, None, x.shape[0], rows, len(counts), K, N)
    assert torch.equal(y.to(R.D), R.matmul(x[src.long()], off, w)[0])
    dx = torch.empty(rows, K, dtype=BF, device="cuda")
    dy = torch.randint(-1, 2, (rows, N), generator=g, device="cuda").to(BF)
    dy[:, 128:] = 0  # (sums below 256)
    T.tpmlp_moe_matmul_dx(dy, off, w, None, dx, rows, len(counts), K, N)
    assert torch.equal(dx.to(R.D), R.matmul(dy, off, w.transpose(1, 2).contiguous())[0])
    dw, db = torch.empty(len(counts), K, N, dtype=F32, device="cuda"), torch.empty(len(counts), N, dtype=F32, device="cuda")
    T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, x.shape[0], rows, len(counts), K, N)
    ref = R.dw(x[src.long()], off, dy, len(counts))
    assert torch.equal(dw.to(R.D), ref[0]) and torch.equal(db.to(R.D), ref[2])


@pytest.mark.parametrize("more", [0, 10])
def test_a_row_is_not_touched_by_its_neighbours(T, more):
    """NaN and infinities in other rows of the same tile, the same expert and the next stay where they are."""
    K, N, counts = 136, 264, [20, 70, 130] + [0] * more
    rows, off, _, x = case(counts, K, False, behind=0)
    w, dy = rnd(3 + more, K, N, seed=2, scale=K**-0.5), rnd(rows, N, seed=4)
    bad = [3, 20, 89, 90, 219]
    x[bad], dy[bad] = NAN, float("inf")
    good = torch.ones(rows, dtype=torch.bool, device="cuda")
    good[bad] = False
    y, dx = torch.empty(rows, N, dtype=BF, device="cuda"), torch.empty(rows, K, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, None, y, None, rows, rows, 3 + more, K, N)
    T.tpmlp_moe_matmul_dx(dy, off, w, None, dx, rows, 3 + more, K, N)
    assert torch.isfinite(y[good]).all() and torch.isnan(y[~good]).all()
    assert torch.isfinite(dx[good]).all() and not torch.isfinite(dx[~good]).any()
    # an expert's weight gradient is of its own rows alone
    x, dy = rnd(rows, K, seed=7), rnd(rows, N, seed=8)
    x[20:90], dy[20:90] = NAN, float("inf")
    dw, db = torch.empty(3 + more, K, N, dtype=F32, device="cuda"), torch.empty(3 + more, N, dtype=F32, device="cuda")
    T.tpmlp_moe_matmul_dw(x, None, off, dy, dw, db, rows, rows, 3 + more, K, N)
    assert torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all() and torch.isnan(dw[1]).all()
    assert torch.isfinite(db[0]).all() and torch.isfinite(db[2]).all()


def gated_slack(g, u, eg, eu):
    """silu' is at most 1.1; ex2 and rcp are within 2^-21 together, the two products two roundings."""
    return 1.1 * eg * (u.abs() + eu) + R.silu(g).abs() * eu + 2.0**-20 * (R.silu(g) * u).abs()


@pytest.mark.parametrize("K,f", [(8, 128), (72, 384), (200, 256), (1032, 640), (4104, 128)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("counts", [COUNTS, FEW, [3, 0, 70], [100, 20, 129, 64, 0]], ids=["many", "few", "three", "middle"])
def test_gated_forward(T, K, f, gather, save, counts):
    rows, off, src, x = case(counts, K, gather, seed=f)
    e, n = len(counts), sum(counts)
    w, b = rnd(e, K, 2 * f, seed=2, scale=1.5 * K**-0.5), rnd(e, 2 * f, seed=3)
    y = torch.full((rows, f), 7.0, dtype=BF, device="cuda")
    h = torch.full((rows, 2 * f), 7.0, dtype=BF, device="cuda") if save else None
    T.tpmlp_moe_matmul(x, src, off, w, b, y, h, x.shape[0], rows, e, K, 2 * f, act=T.ACT_SWIGLU)
    ref, size = R.matmul((x if src is None else x[src.long()])[:n], off, w, b)
    (g, u), (eg, eu) = R.halves(ref), R.halves(R.product_bound(K) * size)
    R.close(y[:n], R.silu(g) * u, gated_slack(g, u, eg, eu), "Y")
    assert (y[n:] == 7.0).all()
    if save:
        R.close(h[:n], ref, R.product_bound(K) * size, "H")
        assert (h[n:] == 7.0).all()


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("out", [BF, F32])
def test_dx(T, K, N, out):
    rows, off, _, dy = case(COUNTS, N, False, seed=K)
    e, n = len(COUNTS), sum(COUNTS)
    w = rnd(e, K, N, seed=2, scale=N**-0.5)
    w[0] = NAN
    dx = torch.full((rows, K), 7.0, dtype=out, device="cuda")
    T.tpmlp_moe_matmul_dx(dy, off, w, None, dx, rows, e, K, N, dx_dt=0 if out == BF else 1)
    ref, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    R.close(dx[:n], ref, R.product_bound(N) * size, "dX")
    assert (dx[n:] == 7.0).all()


@pytest.mark.parametrize("f,N", [(128, 8), (384, 72), (256, 200), (640, 1032)])
def test_gated_dx(T, f, N):
    rows, off, _, dy = case(COUNTS, N, False, seed=f)
    e, n = len(COUNTS), sum(COUNTS)
    w, h = rnd(e, f, N, seed=2, scale=N**-0.5), rnd(rows, 2 * f, seed=3, scale=2.0)
    dh = torch.full((rows, 2 * f), 7.0, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul_dx(dy, off, w, h, dh, rows, e, f, N, act=T.ACT_SWIGLU)
    d, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    g, u = R.halves(h[:n].to(R.D))
    ed = R.product_bound(N) * size
    ref = R.packed(d * u * R.dsilu(g), d * R.silu(g))
    # the approximations (2^-21 of sigma) reach silu' through 1 + g (1 - sigma)
    slack = R.packed(u.abs() * (ed * R.dsilu(g).abs() + d.abs() * 2.0**-20 * (1 + 2 * g.abs())),
                     ed * R.silu(g).abs() + 2.0**-20 * (d * R.silu(g)).abs())
    R.close(dh[:n], ref, slack, "dH")
    assert (dh[n:] == 7.0).all()


@pytest.mark.parametrize("K,N", SHAPES + [(136, 4104), (2056, 72)])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("counts", [COUNTS, FEW, [3, 0, 70], [100, 20, 129, 64, 0], [1]], ids=["many", "few", "three", "middle", "one"])
def test_dx_of_few_and_many_rows(T, K, N, out, counts):
    rows, off, _, dy = case(counts, N, False, seed=K)
    e, n = len(counts), sum(counts)
    dy[n:] = NAN  # rows behind the last
    w = rnd(e, K, N, seed=2, scale=N**-0.5)
    for i in (i for i, c in enumerate(counts) if c == 0):
        w[i] = NAN
    dx = torch.full((rows, K), 7.0, dtype=out, device="cuda")
    T.tpmlp_moe_matmul_dx(dy, off, w, None, dx, rows, e, K, N, dx_dt=0 if out == BF else 1)
    ref, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    R.close(dx[:n], ref, R.product_bound(N) * size, "dX")
    assert (dx[n:] == 7.0).all()


@pytest.mark.parametrize("f,N", [(128, 8), (384, 72), (640, 1032), (128, 4104), (1152, 200), (2048, 72)])
@pytest.mark.parametrize("counts", [COUNTS, FEW, [3, 0, 70], [100, 20, 129, 64, 0], [1]], ids=["many", "few", "three", "middle", "one"])
def test_gated_dx_of_few_and_many_rows(T, f, N, counts):
    rows, off, _, dy = case(counts, N, False, seed=f)
    e, n = len(counts), sum(counts)
    w, h = rnd(e, f, N, seed=2, scale=N**-0.5), rnd(rows, 2 * f, seed=3, scale=2.0)
    dy[n:], h[n:] = NAN, NAN
    for i in (i for i, c in enumerate(counts) if c == 0):
        w[i] = NAN
    dh = torch.full((rows, 2 * f), 7.0, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul_dx(dy, off, w, h, dh, rows, e, f, N, act=T.ACT_SWIGLU)
    d, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    g, u = R.halves(h[:n].to(R.D))
    ed = R.product_bound(N) * size
    # (slack as in test_gated_dx)
    slack = R.packed(u.abs() * (ed * R.dsilu(g).abs() + d.abs() * 2.0**-20 * (1 + 2 * g.abs())),
                     ed * R.silu(g).abs() + 2.0**-20 * (d * R.silu(g)).abs())
    R.close(dh[:n], R.packed(d * u * R.dsilu(g), d * R.silu(g)), slack, "dH")
    assert (dh[n:] == 7.0).all()


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", [BF, F32])
def test_dw(T, K, N, gather, out):
    rows, off, src, x = case(COUNTS, K, gather, seed=K)
    e, n = len(COUNTS), sum(COUNTS)
    dy = rnd(rows, N, seed=4)
    dw, db = (torch.full(s, NAN, dtype=out, device="cuda") for s in ((e, K, N), (e, N)))
    T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, x.shape[0], rows, e, K, N, grad_dt=0 if out == BF else 1)
    ref, size, rb, sb = R.dw((x if src is None else x[src.long()])[:n], off, dy[:n], e)
    R.close(dw, ref, R.product_bound(max(COUNTS)) * size, "dW")
    R.close(db, rb, (max(COUNTS) / 32 + 32) * 2.0**-24 * sb, "dbias")
    assert (dw[0] == 0).all() and (db[5] == 0).all()


# many rows an expert, long contractions and, with the last sizes, enough tiles that rows in order run on two accumulators too
LONG = [[1300, 0, 1801], [2700], [1023, 1090]]


@pytest.mark.parametrize("counts", LONG)
@pytest.mark.parametrize("N", [136, 1032, 2000])
@pytest.mark.parametrize("out", [BF, F32])
def test_many_rows_in_order(T, counts, N, out):
    K, e, n, dt = 4104, len(counts), sum(counts), 0 if out == BF else 1
    rows, off, _, x = case(counts, K, False, seed=N)
    w, b = rnd(e, K, N, seed=2, scale=K**-0.5), rnd(e, N, seed=3)
    y = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, b, y, None, rows, rows, e, K, N, out_dt=dt)
    ref, size = R.matmul(x[:n], off, w, b)
    R.close(y[:n], ref, R.product_bound(K) * size, "Y")
    assert (y[n:] == 7.0).all()
    dx = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    v = w.transpose(1, 2).contiguous()
    T.tpmlp_moe_matmul_dx(x, off, v, None, dx, rows, e, N, K, dx_dt=dt)
    ref, size = R.matmul(x[:n], off, w)
    R.close(dx[:n], ref, R.product_bound(K) * size, "dX")
    assert (dx[n:] == 7.0).all()


@pytest.mark.parametrize("counts", LONG)
@pytest.mark.parametrize("f", [128, 1152])
def test_many_rows_in_order_gated(T, counts, f):
    K, e, n = 4104, len(counts), sum(counts)
    rows, off, _, x = case(counts, K, False, seed=f)
    w, b = rnd(e, K, 2 * f, seed=2, scale=K**-0.5), rnd(e, 2 * f, seed=3)
    y, h = torch.full((rows, f), 7.0, dtype=BF, device="cuda"), torch.full((rows, 2 * f), 7.0, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, b, y, h, rows, rows, e, K, 2 * f, act=T.ACT_SWIGLU)
    ref, size = R.matmul(x[:n], off, w, b)
    R.close(h[:n], ref, R.product_bound(K) * size, "H")
    g, u = R.halves(ref)
    eg, eu = R.halves(R.product_bound(K) * size)
    R.close(y[:n], R.silu(g) * u, gated_slack(g, u, eg, eu), "Y")
    assert (y[n:] == 7.0).all() and (h[n:] == 7.0).all()


@pytest.mark.parametrize("counts", LONG + [[2700, 61], [3, 2900]])
@pytest.mark.parametrize("K,N", [(8, 8), (72, 520), (520, 136), (2056, 1032), (1032, 4616)])
@pytest.mark.parametrize("out", [BF, F32])
def test_many_rows_dw_in_order(T, counts, K, N, out):
    rows, off, _, x = case(counts, K, False, seed=K)
    e, n = len(counts), sum(counts)
    dy = rnd(rows, N, seed=4)
    x[n:], dy[n:] = NAN, NAN  # rows behind the last
    dw, db = (torch.full(s, NAN, dtype=out, device="cuda") for s in ((e, K, N), (e, N)))
    T.tpmlp_moe_matmul_dw(x, None, off, dy, dw, db, rows, rows, e, K, N, grad_dt=0 if out == BF else 1)
    ref, size, rb, sb = R.dw(x[:n], off, dy[:n], e)
    R.close(dw, ref, R.product_bound(max(counts)) * size, "dW")
    R.close(db, rb, (max(counts) / 32 + 32) * 2.0**-24 * sb, "dbias")
    x[off[e - 1]:], dy[off[e - 1]:] = float("inf"), NAN  # of the last expert: the others' stay as they are
    again = torch.full_like(dw, NAN)
    T.tpmlp_moe_matmul_dw(x, None, off, dy, again, None, rows, rows, e, K, N, grad_dt=0 if out == BF else 1)
    assert torch.equal(again[: e - 1], dw[: e - 1])


@pytest.mark.parametrize("K", [8, 72, 200, 1032])
@pytest.mark.parametrize("N", [1544, 1600])
@pytest.mark.parametrize("out", [BF, F32])
def test_gathered_rows_of_many_tiles(T, K, N, out):
    """Enough tiles that gathered rows run on two accumulators."""
    rows, off, src, x = case(COUNTS, K, True, seed=K)
    e, n, dt = len(COUNTS), sum(COUNTS), 0 if out == BF else 1
    w, b, dy = rnd(e, K, N, seed=2, scale=K**-0.5), rnd(e, N, seed=3), rnd(rows, N, seed=4)
    w[0] = NAN  # an expert without rows
    y = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, b, y, None, x.shape[0], rows, e, K, N, out_dt=dt)
    xs = x[src.long()][:n]
    ref, size = R.matmul(xs, off, w, b)
    R.close(y[:n], ref, R.product_bound(K) * size, "Y")
    assert (y[n:] == 7.0).all()
    dw, db = (torch.full(s, NAN, dtype=out, device="cuda") for s in ((e, K, N), (e, N)))
    T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, x.shape[0], rows, e, K, N, grad_dt=dt)
    ref, size, rb, sb = R.dw(xs, off, dy[:n], e)
    R.close(dw, ref, R.product_bound(max(COUNTS)) * size, "dW")
    R.close(db, rb, (max(COUNTS) / 32 + 32) * 2.0**-24 * sb, "dbias")
    assert (dw[0] == 0).all() and (db[5] == 0).all()
    # the last expert with rows reads a token of its own that is not finite: the others' results stay as they are
    last = max(i for i, c in enumerate(COUNTS) if c)
    lo, hi = int(off[last]), int(off[last + 1])
    x2 = torch.cat([x, torch.full((1, K), float("inf"), dtype=BF, device="cuda")])
    src2, dy2 = src.clone(), dy.clone()
    src2[lo:hi], dy2[lo:hi] = x.shape[0], NAN
    y2, dw2 = torch.full_like(y, 7.0), torch.full_like(dw, NAN)
    T.tpmlp_moe_matmul(x2, src2, off, w, b, y2, None, x2.shape[0], rows, e, K, N, out_dt=dt)
    T.tpmlp_moe_matmul_dw(x2, src2, off, dy2, dw2, None, x2.shape[0], rows, e, K, N, grad_dt=dt)
    assert torch.equal(y2[:lo], y[:lo]) and torch.equal(dw2[:last], dw[:last]) and not torch.isfinite(dw2[last]).any()


@pytest.mark.parametrize("K", [8, 200, 1032])
@pytest.mark.parametrize("save", [False, True])
def test_gathered_rows_of_many_tiles_gated(T, K, save):
    f = 896
    rows, off, src, x = case(COUNTS, K, True, seed=K)
    e, n = len(COUNTS), sum(COUNTS)
    w, b = rnd(e, K, 2 * f, seed=2, scale=1.5 * K**-0.5), rnd(e, 2 * f, seed=3)
    y = torch.full((rows, f), 7.0, dtype=BF, device="cuda")
    h = torch.full((rows, 2 * f), 7.0, dtype=BF, device="cuda") if save else None
    T.tpmlp_moe_matmul(x, src, off, w, b, y, h, x.shape[0], rows, e, K, 2 * f, act=T.ACT_SWIGLU)
    ref, size = R.matmul(x[src.long()][:n], off, w, b)
    (g, u), (eg, eu) = R.halves(ref), R.halves(R.product_bound(K) * size)
    R.close(y[:n], R.silu(g) * u, gated_slack(g, u, eg, eu), "Y")
    assert (y[n:] == 7.0).all()
    if save:
        R.close(h[:n], ref, R.product_bound(K) * size, "H")
        assert (h[n:] == 7.0).all()


@pytest.mark.parametrize("counts", [[5], [0, 0, 700], [64, 64], [1] * 100, [0] * 1023 + [40]])
def test_other_distributions(T, counts):
    """One expert, everything on the last, one row each, the most experts."""
    K, N, e = 64, 128, len(counts)
    rows, off, src, x = case(counts, K, True, behind=3)
    w, dy = rnd(e, K, N, seed=2, scale=K**-0.5), rnd(rows, N, seed=4)
    y, dx, dw = torch.zeros(rows, N, dtype=BF, device="cuda"), torch.zeros(rows, K, dtype=BF, device="cuda"), \
        torch.full((e, K, N), NAN, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, None, y, None, x.shape[0], rows, e, K, N)
    T.tpmlp_moe_matmul_dx(dy, off, w, None, dx, rows, e, K, N)
    T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, None, x.shape[0], rows, e, K, N)
    n = sum(counts)
    xs = x[src.long()][:n]
    ref, size = R.matmul(xs, off, w)
    R.close(y[:n], ref, R.product_bound(K) * size, "Y")
    ref, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    R.close(dx[:n], ref, R.product_bound(N) * size, "dX")
    ref, size, _, _ = R.dw(xs, off, dy[:n], e)
    R.close(dw, ref, R.product_bound(max(counts)) * size, "dW")


def test_no_rows(T):
    K, N, e = 64, 128, 3
    w, off = rnd(e, K, N), offsets_of([0, 0, 0])
    T.tpmlp_moe_matmul(None, None, off, w, None, None, None, 0, 0, e, K, N)
    dw, db = torch.full((e, K, N), NAN, device="cuda"), torch.full((e, N), NAN, device="cuda")
    T.tpmlp_moe_matmul_dw(None, None, off, None, dw, db, 0, 0, e, K, N)
    assert (dw == 0).all() and (db == 0).all()
    # rows, but none of any expert
    x, y = rnd(5, K), torch.full((5, N), 3.0, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, None, y, None, 5, 5, e, K, N)
    assert (y == 3.0).all()


def test_a_plan_outside_of_the_rows_is_cut_and_reported(T):
    """Ranges and tokens are compared with their tensors in the kernels, before anything is read through them."""
    K, N = 64, 128
    x, w = rnd(8, K), rnd(2, K, N)
    y = torch.zeros(8, N, dtype=BF, device="cuda")
    off = torch.tensor([0, 6, 9], dtype=I32, device="cuda")  # a row too many
    T.tpmlp_moe_matmul(x, None, off, w, None, y, None, 8, 8, 2, K, N)
    assert T.tpmlp_device_status(check=False) == T.ERR_DEVICE
    ref, size = R.matmul(x, torch.tensor([0, 6, 8]), w)
    R.close(y, ref, R.product_bound(K) * size, "Y")
    src = torch.tensor([0, 1, 2, 3, 4, 5, 8, -1], dtype=I32, device="cuda")  # 8 and -1: no such tokens
    y.zero_()
    T.tpmlp_moe_matmul(x, src, torch.tensor([0, 6, 8], dtype=I32, device="cuda"), w, None, y, None, 8, 8, 2, K, N)
    assert T.tpmlp_device_status(check=False) == T.ERR_DEVICE
    R.close(y[:6], ref[:6], R.product_bound(K) * size[:6], "Y")
    assert T.tpmlp_device_status(check=False) == T.OK


# ------------------------------------------------------------------ combination
@pytest.mark.parametrize("t,k,h", [(1, 1, 8), (4, 2, 5120), (33, 3, 72), (100, 8, 2056), (257, 32, 264), (2000, 2, 136)])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine_and_backward(T, t, k, h, weighted):
    g = torch.Generator(device="cuda").manual_seed(t)
    gone = torch.rand(t, k, generator=g, device="cuda") < 0.2
    rows = t * k + 5
    sr = torch.randperm(rows, generator=g, device="cuda")[: t * k].view(t, k).int()
    sr = torch.where(gone, -1, sr)
    if t > 3:
        sr[3] = -1  # a token without rows
    o, dz = rnd(rows, h, seed=1), rnd(t, h, seed=2)
    used = torch.zeros(rows, dtype=torch.bool, device="cuda")
    used[sr[sr >= 0].long()] = True
    o[~used] = NAN  # rows of no slot
    w = torch.rand(t, k, generator=g, device="cuda") if weighted else None
    if weighted:
        w[sr < 0] = NAN  # weights of no row
    z, do, dw = torch.full((t, h), NAN, dtype=BF, device="cuda"), torch.full((rows, h), 7.0, dtype=BF, device="cuda"), \
        torch.full((t, k), NAN, device="cuda")
    T.tpmlp_moe_combine(o, sr, w, z, t, rows, k, h)
    ref, size = R.combine(o, sr, w)
    R.close(z, ref, k * 2.0**-23 * size, "Z")
    T.tpmlp_moe_combine_bwd(o, sr, w, dz, do, dw, t, rows, k, h)
    assert (do[~used] == 7.0).all()
    at = sr.clamp(min=0).long()
    there = (sr >= 0)[:, :, None]
    prod = torch.where(there, o[at].to(R.D) * dz.to(R.D)[:, None], torch.zeros((), dtype=R.D, device="cuda"))
    # a lane adds h / 256 + 1 groups of 8 products, then 5 sums across lanes
    R.close(dw, prod.sum(2), (h / 32 + 32) * 2.0**-24 * prod.abs().sum(2), "dweights")
    ww = (torch.ones(t, k, device="cuda") if w is None else w)[:, :, None].to(R.D) * dz.to(R.D)[:, None]
    R.close(do[sr[sr >= 0].long()], ww[sr >= 0], 2.0**-24 * ww[sr >= 0].abs(), "dO")
    if weighted:
        do2 = torch.full_like(do, 7.0)
        T.tpmlp_moe_combine_bwd(None, sr, w, dz, do2, None, t, rows, k, h)
        assert torch.equal(do, do2)


def test_combine_without_rows(T):
    sr = torch.full((3, 2), -1, dtype=I32, device="cuda")
    z, dw = torch.full((3, 64), NAN, dtype=BF, device="cuda"), torch.full((3, 2), NAN, device="cuda")
    T.tpmlp_moe_combine(None, sr, None, z, 3, 0, 2, 64)
    T.tpmlp_moe_combine_bwd(None, sr, None, rnd(3, 64), None, dw, 3, 0, 2, 64)
    assert (z == 0).all() and (dw == 0).all()
