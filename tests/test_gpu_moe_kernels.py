"""Grouped products on the GPU, each kernel (tests/moe_cases.py; tests/test_moe_choice_host.py checks that it is the one that
runs), against 64 bits (tests/moe_ref.py): few and many experts, skewed plans, up to 1024 experts."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import moe_cases as C  # noqa: E402
import moe_ref as R  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN = float("nan")


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the cases are for 152 SMs")
    from megatron_tensor_mlp_gb300 import tpmlp
    yield tpmlp
    tpmlp.tpmlp_device_status()


def rnd(*shape, seed=0, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def gated_slack(g, u, eg, eu):
    """silu' is at most 1.1; ex2 and rcp are within 2^-21 together, the two products two roundings."""
    return 1.1 * eg * (u.abs() + eu) + R.silu(g).abs() * eu + 2.0**-20 * (R.silu(g) * u).abs()


@pytest.mark.parametrize("case", C.CASES, ids=C.name)
def test_kernel(T, case):
    op, _, counts, behind, K, N, gathered = case
    e, n = len(counts), sum(counts)
    rows = n + behind
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=I32, device="cuda")
    long = N if "dx" in op else K
    tokens = max(rows // 2, 1) if gathered else rows
    x = rnd(tokens, long, seed=1)  # (dx: dY)
    src = None
    if gathered:
        g = torch.Generator(device="cuda").manual_seed(2)
        src = torch.randint(0, tokens, (rows,), generator=g, device="cuda", dtype=I32)
    else:
        x[n:] = NAN  # rows behind the last
    xs = (x if src is None else x[src.long()])[:n]
    if op != "dw":
        w = rnd(e, K, N, seed=3, scale=long**-0.5)
        w[torch.tensor(counts, device="cuda") == 0] = NAN  # experts without rows
    if op == "forward":
        b = rnd(e, N, seed=4)
        for out in (BF, F32):
            y = torch.full((rows, N), 7.0, dtype=out, device="cuda")
            T.tpmlp_moe_matmul(x, src, off, w, b, y, None, tokens, rows, e, K, N, out_dt=0 if out == BF else 1)
            ref, size = R.matmul(xs, off, w, b)
            R.close(y[:n], ref, R.product_bound(K) * size, "Y")
            assert (y[n:] == 7.0).all()
    elif op == "gated":
        b, f = rnd(e, N, seed=4), N // 2
        y, h = torch.full((rows, f), 7.0, dtype=BF, device="cuda"), torch.full((rows, N), 7.0, dtype=BF, device="cuda")
        T.tpmlp_moe_matmul(x, src, off, w, b, y, h, tokens, rows, e, K, N, act=T.ACT_SWIGLU)
        ref, size = R.matmul(xs, off, w, b)
        (gate, up), (eg, eu) = R.halves(ref), R.halves(R.product_bound(K) * size)
        R.close(y[:n], R.silu(gate) * up, gated_slack(gate, up, eg, eu), "Y")
        R.close(h[:n], ref, R.product_bound(K) * size, "H")
        assert (y[n:] == 7.0).all() and (h[n:] == 7.0).all()
        again = torch.full_like(y, 7.0)
        T.tpmlp_moe_matmul(x, src, off, w, b, again, None, tokens, rows, e, K, N, act=T.ACT_SWIGLU)
        assert torch.equal(again, y)
    elif op == "dx":
        for out in (BF, F32):
            dx = torch.full((rows, K), 7.0, dtype=out, device="cuda")
            T.tpmlp_moe_matmul_dx(x, off, w, None, dx, rows, e, K, N, dx_dt=0 if out == BF else 1)
            ref, size = R.matmul(xs, off, w.transpose(1, 2))
            R.close(dx[:n], ref, R.product_bound(N) * size, "dX")
            assert (dx[n:] == 7.0).all()
    elif op == "gated dx":
        h = rnd(rows, 2 * K, seed=5, scale=2.0)
        h[n:] = NAN
        dh = torch.full((rows, 2 * K), 7.0, dtype=BF, device="cuda")
        T.tpmlp_moe_matmul_dx(x, off, w, h, dh, rows, e, K, N, act=T.ACT_SWIGLU)
        d, size = R.matmul(xs, off, w.transpose(1, 2))
        gate, up = R.halves(h[:n].to(R.D))
        ed = R.product_bound(N) * size
        # the approximations (2^-21 of sigma) reach silu' through 1 + g (1 - sigma)
        slack = R.packed(up.abs() * (ed * R.dsilu(gate).abs() + d.abs() * 2.0**-20 * (1 + 2 * gate.abs())),
                         ed * R.silu(gate).abs() + 2.0**-20 * (d * R.silu(gate)).abs())
        R.close(dh[:n], R.packed(d * up * R.dsilu(gate), d * R.silu(gate)), slack, "dH")
        assert (dh[n:] == 7.0).all()
    else:
        dy = rnd(rows, N, seed=6)
        dy[n:] = NAN
        ref, size, rb, sb = R.dw(xs, off, dy[:n], e)
        for out in (BF, F32):
            dw, db = (torch.full(s, NAN, dtype=out, device="cuda") for s in ((e, K, N), (e, N)))
            T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, tokens, rows, e, K, N, grad_dt=0 if out == BF else 1)
            R.close(dw, ref, R.product_bound(max(counts)) * size, "dW")
            R.close(db, rb, (max(counts) / 32 + 32) * 2.0**-24 * sb, "dbias")


def test_a_layer_of_many_small_experts(T):
    """8 of 256 experts of 768 features on 1000 tokens, some of them padding, one expert that nobody chooses: routing, both
    products and the combination, each against 64 bits on the inputs that the one ahead of it gave."""
    t, k, e, h, f = 1000, 8, 256, 512, 768
    x, logits = rnd(t, h, seed=1), rnd(t, e, seed=2, dtype=F32)
    logits[::50] = -float("inf")
    logits[:, 17] = -float("inf")
    w1, w2 = rnd(e, h, 2 * f, seed=3, scale=h**-0.5), rnd(e, f, h, seed=4, scale=f**-0.5)
    new = lambda *s, dtype=BF: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    ids, w, off, rt, sr = new(t, k, dtype=I32), new(t, k, dtype=F32), new(e + 1, dtype=I32), new(t * k, dtype=I32), new(t, k, dtype=I32)
    ws = new(T.tpmlp_moe_route_ws_bytes(t, e, k), dtype=torch.uint8)
    y, hh, o, z = new(t * k, f), new(t * k, 2 * f), new(t * k, h), new(t, h)
    T.tpmlp_moe_route(logits, ids, w, off, rt, sr, ws, t, e, k, dt=T.F32)
    T.tpmlp_moe_matmul(x, rt, off, w1, None, y, hh, t, t * k, e, h, 2 * f, act=T.ACT_SWIGLU)
    T.tpmlp_moe_matmul(y, None, off, w2, None, o, None, t * k, t * k, e, f, h)
    T.tpmlp_moe_combine(o, sr, w, z, t, t * k, k, h)
    plan = R.route(logits.cpu(), k, 1)
    for got, want in zip((ids, off, rt, sr), (plan[0], *plan[2:])):
        assert torch.equal(got.cpu(), want)
    n = int(off[-1])
    assert n == (t - len(range(0, t, 50))) * k and off[17] == off[18]
    ref, size = R.matmul(x[rt[:n].long()], off, w1)
    (gate, up), (eg, eu) = R.halves(ref), R.halves(R.product_bound(h) * size)
    R.close(hh[:n], ref, R.product_bound(h) * size, "H")
    R.close(y[:n], R.silu(gate) * up, gated_slack(gate, up, eg, eu), "Y")
    ref, size = R.matmul(y[:n], off, w2)
    R.close(o[:n], ref, R.product_bound(f) * size, "O")
    ref, size = R.combine(o, sr, w)
    R.close(z, ref, k * 2.0**-23 * size, "Z")
    assert (z[::50] == 0).all()


@pytest.mark.parametrize("case", C.CASES, ids=C.name)
def test_kernel_without_rows_and_with_rows_of_nobody_ahead(T, case):
    """Plans that leave every expert empty, at either end of the rows: outputs stay as they were, weight gradients are zero.
    And one whose first range starts behind rows that no expert has."""
    op, _, counts, behind, K, N, gathered = case
    e, rows = len(counts), sum(counts) + behind
    long = N if "dx" in op else K
    tokens = max(rows // 2, 1) if gathered else rows
    x = rnd(tokens, long, seed=1)
    src = torch.arange(rows, dtype=I32, device="cuda") % tokens if gathered else None
    w = None if op == "dw" else rnd(e, K, N, seed=3, scale=long**-0.5)
    other = rnd(rows, 2 * K if op == "gated dx" else N, seed=5)  # H, dY

    def call(off):
        new = lambda *s, dtype=BF: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
        if op == "forward":
            out = [new(rows, N)]
            T.tpmlp_moe_matmul(x, src, off, w, None, *out, None, tokens, rows, e, K, N)
        elif op == "gated":
            out = [new(rows, N // 2), new(rows, N)]
            T.tpmlp_moe_matmul(x, src, off, w, None, *out, tokens, rows, e, K, N, act=T.ACT_SWIGLU)
        elif op == "dx":
            out = [new(rows, K)]
            T.tpmlp_moe_matmul_dx(x, off, w, None, *out, rows, e, K, N)
        elif op == "gated dx":
            out = [new(rows, 2 * K)]
            T.tpmlp_moe_matmul_dx(x, off, w, other, *out, rows, e, K, N, act=T.ACT_SWIGLU)
        else:
            out = [new(e, K, N, dtype=F32), new(e, N, dtype=F32)]
            T.tpmlp_moe_matmul_dw(x, src, off, other, *out, tokens, rows, e, K, N)
        return out

    for at in (0, rows):
        for o in call(torch.full((e + 1,), at, dtype=I32, device="cuda")):
            assert (o == (0.0 if op == "dw" else 7.0)).all()
    # the last rows on two experts, those ahead on none
    first = rows - min(rows, 41)
    mid = (first + rows) // 2
    off = torch.tensor([first] * (e // 2 + 1) + [mid] * (e - e // 2 - 1) + [rows], dtype=I32, device="cuda")
    off = off[: e + 1] if e > 1 else torch.tensor([first, rows], dtype=I32, device="cuda")
    off[-1] = rows
    got = call(off)
    if op == "dw":
        xs = x if src is None else x[src.long()]
        ref, size, rb, sb = R.dw(xs, off, other, e)
        R.close(got[0], ref, R.product_bound(41) * size, "dW")
        R.close(got[1], rb, 64 * 2.0**-24 * sb, "dbias")
    else:
        for o in got:
            assert (o[:first] == 7.0).all() and not (o[first:] == 7.0).all(1).any()
    assert T.tpmlp_device_status(check=False) == T.OK
