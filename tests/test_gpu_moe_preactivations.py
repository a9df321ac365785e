"""The gated experts with their pre-activations saved in fp32, on the GPU, against 64 bits (tests/moe_ref.py)."""
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
    from megatron_tensor_mlp_gb300 import tpmlp
    yield tpmlp
    tpmlp.tpmlp_device_status()


def rnd(*shape, seed=0, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def plan(case):
    op, _, counts, behind, K, N, gathered = case
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=I32, device="cuda")
    return len(counts), sum(counts), sum(counts) + behind, off


@pytest.mark.parametrize("case", [c for c in C.CASES if c[0] == "gated"], ids=C.name)
@pytest.mark.parametrize("biased", [True, False])
def test_saved_in_fp32(T, case, biased):
    """H to fp32's bound, Y to the bit of a call that saves nothing."""
    _, _, counts, _, K, N, gathered = case
    e, n, rows, off = plan(case)
    tokens = max(rows // 2, 1) if gathered else rows
    x, w, b = rnd(tokens, K, seed=1), rnd(e, K, N, seed=3, scale=K**-0.5), rnd(e, N, seed=4) if biased else None
    src = None
    if gathered:
        src = torch.randint(0, tokens, (rows,), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=I32)
    y, y0 = (torch.full((rows, N // 2), 7.0, dtype=BF, device="cuda") for _ in range(2))
    h = torch.full((rows, N), 7.0, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, b, y, h, tokens, rows, e, K, N, act=T.ACT_SWIGLU_H32)
    T.tpmlp_moe_matmul(x, src, off, w, b, y0, None, tokens, rows, e, K, N, act=T.ACT_SWIGLU_H32)
    assert torch.equal(y, y0)
    T.tpmlp_moe_matmul(x, src, off, w, b, y0, None, tokens, rows, e, K, N, act=T.ACT_SWIGLU)
    assert torch.equal(y, y0)
    ref, size = R.matmul((x if src is None else x[src.long()])[:n], off, w, b)
    R.close(h[:n], ref, R.product_bound(K) * size, "H")
    assert (h[n:] == 7.0).all() and (y[n:] == 7.0).all()
    half = torch.empty(rows, N, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, src, off, w, b, y0, half, tokens, rows, e, K, N, act=T.ACT_SWIGLU)
    assert torch.equal(h[:n].to(BF), half[:n])


@pytest.mark.parametrize("case", [c for c in C.CASES if c[0] == "gated dx"], ids=C.name)
def test_gradient_from_fp32(T, case):
    _, _, counts, _, K, N, _ = case
    e, n, rows, off = plan(case)
    dy, w, h = rnd(rows, N, seed=1), rnd(e, K, N, seed=3, scale=N**-0.5), rnd(rows, 2 * K, seed=5, scale=2.0, dtype=F32)
    dy[n:], h[n:] = NAN, NAN
    w[torch.tensor(counts, device="cuda") == 0] = NAN
    dh = torch.full((rows, 2 * K), 7.0, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul_dx(dy, off, w, h, dh, rows, e, K, N, act=T.ACT_SWIGLU_H32)
    d, size = R.matmul(dy[:n], off, w.transpose(1, 2))
    gate, up = R.halves(h[:n].to(R.D))
    ed = R.product_bound(N) * size
    # the approximations (2^-21 of sigma) reach silu' through 1 + g (1 - sigma)
    slack = R.packed(up.abs() * (ed * R.dsilu(gate).abs() + d.abs() * 2.0**-20 * (1 + 2 * gate.abs())),
                     ed * R.silu(gate).abs() + 2.0**-20 * (d * R.silu(gate)).abs())
    R.close(dh[:n], R.packed(d * up * R.dsilu(gate), d * R.silu(gate)), slack, "dH")
    assert (dh[n:] == 7.0).all()
    # values that bf16 holds: the bits of the call that takes them so
    dh2 = torch.full_like(dh, 7.0)
    T.tpmlp_moe_matmul_dx(dy, off, w, h.to(BF).float(), dh, rows, e, K, N, act=T.ACT_SWIGLU_H32)
    T.tpmlp_moe_matmul_dx(dy, off, w, h.to(BF), dh2, rows, e, K, N, act=T.ACT_SWIGLU)
    assert torch.equal(dh[:n], dh2[:n])


@pytest.mark.parametrize("rows,h,f", [(512, 1024, 1024), (700, 520, 384), (2048, 1024, 768)])
def test_a_gated_expert_s_gradients_within_the_library_s_bound(T, rows, h, f):
    """Forward and backward of the two layers in bf16: 3e-3 in the Frobenius norm, the bound of the gated block on dense weights.
    dY, a product and a rounding to bf16 per layer, is what separates dX from 64 bits: sqrt(2) 1.7e-3 = 2.4e-3, with H in bf16
    3.0e-3."""
    x, do = rnd(rows, h, seed=1), rnd(rows, h, seed=2)
    w1, w2 = rnd(2, h, 2 * f, seed=3, scale=h**-0.5), rnd(2, f, h, seed=4, scale=f**-0.5)
    off = torch.tensor([0, rows // 3, rows], dtype=I32, device="cuda")
    new = lambda *s, dtype=BF: torch.full(s, NAN, dtype=dtype, device="cuda")  # noqa: E731
    y, hh, dh, dx = new(rows, f), new(rows, 2 * f, dtype=F32), new(rows, 2 * f), new(rows, h)
    dw1, dw2 = new(2, h, 2 * f, dtype=F32), new(2, f, h, dtype=F32)
    T.tpmlp_moe_matmul(x, None, off, w1, None, y, hh, rows, rows, 2, h, 2 * f, act=T.ACT_SWIGLU_H32)
    T.tpmlp_moe_matmul_dx(do, off, w2, hh, dh, rows, 2, f, h, act=T.ACT_SWIGLU_H32)
    T.tpmlp_moe_matmul_dx(dh, off, w1, None, dx, rows, 2, h, 2 * f)
    T.tpmlp_moe_matmul_dw(x, None, off, dh, dw1, None, rows, rows, 2, h, 2 * f)
    T.tpmlp_moe_matmul_dw(y, None, off, do, dw2, None, rows, rows, 2, f, h)
    gate, up = R.halves(R.matmul(x, off, w1)[0])
    d = R.matmul(do, off, w2.transpose(1, 2))[0]
    rdh = R.packed(d * up * R.dsilu(gate), d * R.silu(gate))
    refs = {"dX": (dx, R.matmul(rdh, off, w1.to(R.D).transpose(1, 2))[0]), "dW1": (dw1, R.dw(x, off, rdh, 2)[0]),
            "dW2": (dw2, R.dw(R.silu(gate) * up, off, do, 2)[0])}
    for name, (got, ref) in refs.items():
        rel = float((got.to(R.D) - ref).norm() / ref.norm())
        assert rel <= (2.6e-3 if name == "dX" else 2e-3), (name, rel)


def rounded(v):
    return v.to(F32).to(BF).to(R.D)


@pytest.mark.parametrize("t,h,f,e,k", [(37, 136, 128, 8, 3), (300, 256, 384, 16, 2), (1000, 512, 256, 8, 2)])
def test_a_layer_rounds_where_it_says(T, t, h, f, e, k):
    """The example layer against the same chain in 64 bits with its roundings to bf16 (n, logits, Y, O, Z; dO, dH, dR, dn's two
    parts and their sum, dlogits, dX): what is left is fp32's error, and roundings that it tips over.  A value within 2^-16 of itself
    of the middle of two bf16 neighbours, 2^-8 apart or more, may go either way (the sums of up to 1000 terms are that good):
    one in 2^7 of them, by 2^-8: 2^-8 2^-3.5 in the root mean square, at 14 places on the way: sqrt(14) 2^-11.5 = 1.3e-3 of a
    result (roundings alone make 4e-3 to 5e-3 of it)."""
    import test_gpu_moe_block as B
    layer, w = B.layer_of(h, f, e, k)
    X, dZ = rnd(t, h, seed=20), rnd(t, h, seed=21)
    Z, saved = layer.forward(X, save=True)
    got = (Z, *layer.backward(saved, dZ))
    gamma, beta, router, gate, up, down = (v.to(R.D) for v in w)
    ids = saved[5].long()
    x = X.to(R.D)
    y0, mean, rstd = R.norm(X, w[0], w[1], 1e-5)
    n = rounded(y0)
    logits = rounded(n @ router)
    p = torch.softmax(logits.gather(1, ids), 1)
    z, dn, dwt = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(p)
    dG, dU, dD = torch.zeros_like(gate), torch.zeros_like(up), torch.zeros_like(down)
    for j in range(k):
        for i in range(e):
            at = (ids[:, j] == i).nonzero()[:, 0]
            if at.numel() == 0:
                continue
            v, c = n[at], p[at, j, None]
            g, u = v @ gate[i], v @ up[i]
            y = rounded(R.silu(g) * u)
            o = rounded(y @ down[i])
            z[at] += c * o
            dz = dZ[at].to(R.D)
            dwt[at, j] = (dz * o).sum(1)
            do = rounded(c * dz)
            dy = do @ down[i].t()
            dg, du = rounded(dy * u * R.dsilu(g)), rounded(dy * R.silu(g))
            dn[at] += rounded(dg @ gate[i].t() + du @ up[i].t())
            dG[i] += v.t() @ dg
            dU[i] += v.t() @ du
            dD[i] += y.t() @ do
    inner = (p * dwt).sum(1, keepdim=True)
    dl = rounded(torch.zeros_like(logits).scatter_(1, ids, p * (dwt - inner)))
    dn = rounded(rounded(dn) + rounded(dl @ router.t()))
    dx, dgamma, dbeta = R.norm_bwd(X, w[0], mean, rstd, dn)
    for name, a, b in zip(("Z", "dX", "gamma", "beta", "router", "gate", "up", "down"), got,
                          (rounded(z), rounded(dx), dgamma, dbeta, n.t() @ dl, dG, dU, dD)):
        rel = float((a.to(R.D) - b).norm() / b.norm())
        assert rel <= 14**0.5 * 2.0**-11.5, (name, rel)
