"""The expert operators as a layer runs them: forward and backward against autograd in 64 bits, captured into a graph,
on other streams, two at a time, and at offsets past 32 bits."""
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


def layer_of(h, f, e, k, seed=0):
    from megatron_tensor_mlp_gb300.moe_block import ExpertLayer
    w = [1 + rnd(h, seed=seed, scale=0.1), rnd(h, seed=seed + 1, scale=0.1), rnd(h, e, seed=seed + 2, scale=h**-0.5),
         rnd(e, h, f, seed=seed + 3, scale=h**-0.5), rnd(e, h, f, seed=seed + 4, scale=h**-0.5), rnd(e, f, h, seed=seed + 5, scale=f**-0.5)]
    return ExpertLayer(*w, k), w


def reference(w, k, X, dZ, ids):
    """The layer and its gradients by autograd in 64 bits, on the experts that the kernels chose."""
    leaves = [t.to(R.D).requires_grad_() for t in (X, *w)]
    x, gamma, beta, router, gate, up, down = leaves
    mean = x.mean(1, keepdim=True)
    n = (x - mean) / torch.sqrt((x - mean).square().mean(1, keepdim=True) + 1e-5) * gamma + beta
    p = torch.softmax((n @ router).gather(1, ids.long()), 1)
    z = torch.zeros_like(x)
    for j in range(k):
        for e in range(router.shape[1]):
            at = (ids[:, j] == e).nonzero()[:, 0]
            if at.numel():
                v = n[at]
                z = z.index_add(0, at, p[at, j, None] * ((torch.nn.functional.silu(v @ gate[e]) * (v @ up[e])) @ down[e]))
    return z.detach(), torch.autograd.grad(z, leaves, dZ.to(R.D))


@pytest.mark.parametrize("t,h,f,e,k", [(1, 64, 128, 8, 2), (37, 136, 128, 8, 3), (300, 256, 384, 16, 2), (1500, 512, 256, 8, 2)])
def test_layer_and_gradients(T, t, h, f, e, k):
    layer, w = layer_of(h, f, e, k)
    X, dZ = rnd(t, h, seed=20), rnd(t, h, seed=21)
    Z, saved = layer.forward(X, save=True)
    got = layer.backward(saved, dZ)
    ids, logits = saved[5], saved[4]
    assert torch.equal(torch.sort(logits.float().gather(1, ids.long()), 1, descending=True).values,
                       torch.sort(logits.float(), 1, descending=True).values[:, :k])
    z, grads = reference(w, k, X, dZ, ids)
    # Roundings to bf16 on the way, each off by at most 2^-8 of its value: n, logits, H, Y, O, Z forward; dO, dH, dR, dn (three:
    # two parts and their sum), dlogits and the result backward, on top of the forward's.  A relative error of independent
    # parts passes through a product of random factors unchanged, and sums of n, logits .. are at most their number times 2^-8;
    # a logit of size 3 moves its weight by 3 2^-8 of itself.
    for name, a, b, roundings in (("Z", Z, z, 6 + 3), *((n, a, b, 6 + 3 + 8) for n, a, b in
                                                     zip(("dX", "gamma", "beta", "router", "gate", "up", "down"), got, grads))):
        rel = float((a.to(R.D) - b).norm() / b.norm())
        assert rel <= roundings * 2.0**-8, (name, rel)
    assert torch.equal(layer.forward(X), Z)  # and without saving


def test_layer_of_no_tokens(T):
    layer, _ = layer_of(64, 128, 8, 2)
    X = rnd(0, 64)
    Z, saved = layer.forward(X, save=True)
    dX, *grads = layer.backward(saved, X)
    assert Z.shape == (0, 64) and dX.shape == (0, 64) and all(float(g.abs().sum()) == 0 for g in grads)


def test_layer_refuses_other_tensors(T):
    layer, w = layer_of(64, 128, 8, 2)
    for bad in (rnd(5, 72), rnd(5, 64, dtype=F32), rnd(64, 5).t(), rnd(5, 64).cpu()):
        with pytest.raises(ValueError):
            layer.forward(bad)
    with pytest.raises(ValueError):
        layer.load(*w[:5], w[5].transpose(1, 2))


def test_example_runs(T):
    from megatron_tensor_mlp_gb300.moe_block import train_and_serve
    losses, served, batch = train_and_serve(tokens=128, steps=3)
    assert len(losses) == 3 and all(v == v for v in losses)
    # the same products in another order of additions, rounded to bf16 six times on the way
    assert float((served.to(R.D) - batch.to(R.D)).norm() / batch.to(R.D).norm()) <= 6 * 2.0**-8


def test_captured_and_replayed_on_new_inputs(T):
    """A graph of forward and backward, replayed on other tokens (other plans): the bits of eager calls."""
    layer, _ = layer_of(256, 128, 8, 2)
    X, dZ = rnd(200, 256, seed=1), rnd(200, 256, seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _, saved = layer.forward(X, save=True)
            layer.backward(saved, dZ)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z, saved = layer.forward(X, save=True)
        grads = layer.backward(saved, dZ)
    for seed in (11, 12):
        X.copy_(rnd(200, 256, seed=seed))
        dZ.copy_(rnd(200, 256, seed=seed + 5))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (Z, *grads)]
        Z1, saved1 = layer.forward(X, save=True)
        for a, b in zip(got, (Z1, *layer.backward(saved1, dZ))):
            assert torch.equal(a, b)


def test_two_calls_at_once(T):
    """Two layers on two streams, their kernels interleaved, give what each gives alone."""
    pairs = [layer_of(256, 128, 8, 2, seed=s)[0] for s in (0, 50)]
    X = [rnd(333, 256, seed=s) for s in (3, 4)]
    dZ = [rnd(333, 256, seed=s) for s in (5, 6)]

    def alone(i):
        Z, saved = pairs[i].forward(X[i], save=True)
        return [Z, *pairs[i].backward(saved, dZ[i])]

    want = [alone(0), alone(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(alone(i))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_same_bits_every_time(T):
    layer, _ = layer_of(512, 256, 16, 4)
    X, dZ = rnd(700, 512, seed=1), rnd(700, 512, seed=2)
    outs = []
    for _ in range(3):
        Z, saved = layer.forward(X, save=True)
        outs.append([Z, *layer.backward(saved, dZ)])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


# ------------------------------------------------------------------ tensors of more than 2^31 elements
def test_offsets_past_32_bits_rows(T):
    """Rows behind element 2^31 of X, Y, dY and dX, in order and gathered."""
    K, N, rows, e = 8, 131072, 16600, 2
    assert rows * N > 2**31
    off = torch.tensor([0, 150, rows], dtype=I32, device="cuda")
    x, w = rnd(rows, K), rnd(e, K, N, seed=2)
    y = torch.empty(rows, N, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, None, y, None, rows, rows, e, K, N)
    at = torch.tensor([0, 149, 150, 16383, 16384, rows - 1], device="cuda")
    ref, size = x[at].to(R.D) @ w[1].to(R.D), x[at].to(R.D).abs() @ w[1].to(R.D).abs()
    ref[:2], size[:2] = x[at[:2]].to(R.D) @ w[0].to(R.D), x[at[:2]].to(R.D).abs() @ w[0].to(R.D).abs()
    R.close(y[at], ref, R.product_bound(K) * size, "Y")
    dx = torch.empty(rows, K, dtype=BF, device="cuda")  # Y as the gradient
    T.tpmlp_moe_matmul_dx(y, off, w, None, dx, rows, e, K, N)
    pick = [w[0]] * 2 + [w[1]] * 4
    ref = torch.stack([y[r].to(R.D) @ v.to(R.D).t() for r, v in zip(at, pick)])
    size = torch.stack([y[r].to(R.D).abs() @ v.to(R.D).abs().t() for r, v in zip(at, pick)])
    R.close(dx[at], ref, R.product_bound(N) * size, "dX")
    # gathered from behind 2^31, contracted over the long side
    v, src = rnd(e, N, K, seed=3), torch.tensor([rows - 1, 16384, 0, 5] * 5, dtype=I32, device="cuda")
    few = torch.tensor([0, 9, 20], dtype=I32, device="cuda")
    o = torch.empty(20, K, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(y, src, few, v, None, o, None, rows, 20, e, N, K)
    ref, size = R.matmul(y[src.long()], few, v)
    R.close(o, ref, R.product_bound(N) * size, "gathered")
    dw, db = torch.empty(e, N, K, dtype=BF, device="cuda"), torch.empty(e, K, dtype=BF, device="cuda")
    d = rnd(20, K, seed=4)
    T.tpmlp_moe_matmul_dw(y, src, few, d, dw, db, rows, 20, e, N, K, grad_dt=0)
    ref, size, _, _ = R.dw(y[src.long()], few, d, e)
    R.close(dw, ref, R.product_bound(20) * size, "dW")


def test_offsets_past_32_bits_weights(T):
    """The last of 40 experts' weights and gradients lie behind element 2^31."""
    K, N, e = 4096, 16384, 40
    assert e * K * N > 2**31
    w = torch.zeros(e, K, N, dtype=BF, device="cuda")
    w[-1] = rnd(K, N, seed=2, scale=K**-0.5)
    counts = [0] * (e - 1) + [70]
    off = torch.tensor([0] * e + [70], dtype=I32, device="cuda")
    assert len(counts) == e
    x, y = rnd(70, K), torch.empty(70, N, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, off, w, None, y, None, 70, 70, e, K, N)
    R.close(y, x.to(R.D) @ w[-1].to(R.D), R.product_bound(K) * (x.to(R.D).abs() @ w[-1].to(R.D).abs()), "Y")
    dx = torch.empty(70, K, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul_dx(y, off, w, None, dx, 70, e, K, N)
    R.close(dx, y.to(R.D) @ w[-1].to(R.D).t(), R.product_bound(N) * (y.to(R.D).abs() @ w[-1].to(R.D).abs().t()), "dX")
    w.fill_(NAN)  # now its gradient
    T.tpmlp_moe_matmul_dw(x, None, off, y, w, None, 70, 70, e, K, N, grad_dt=0)
    assert (w[:-1] == 0).all()
    R.close(w[-1], x.to(R.D).t() @ y.to(R.D), R.product_bound(70) * (x.to(R.D).abs().t() @ y.to(R.D).abs()), "dW")


def test_offsets_past_32_bits_norm_and_combine(T):
    rows, h = 2**31 // 4096 + 40, 4096
    x = torch.zeros(rows, h, dtype=BF, device="cuda")
    at = torch.tensor([0, 2**31 // 4096 - 1, 2**31 // 4096, rows - 1], device="cuda")
    x[at] = rnd(4, h, seed=1)
    y = torch.empty_like(x)
    T.tpmlp_layernorm_fwd(x, None, None, y, None, None, rows, h, h, h)
    ref, _, _ = R.norm(x[at], None, None, 1e-5)
    R.close(y[at], ref, 2.0**-16, "y")
    z = torch.empty(4, h, dtype=BF, device="cuda")
    T.tpmlp_moe_combine(x, at.int().view(4, 1), None, z, 4, rows, 1, h)
    assert torch.equal(z, x[at])
    T.tpmlp_moe_combine_bwd(None, at.int().view(4, 1), None, rnd(4, h, seed=9), y, None, 4, rows, 1, h)
    assert torch.equal(y[at], rnd(4, h, seed=9))
