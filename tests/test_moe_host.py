"""Layer norm, routing, grouped products and the combination on the host: workspace sizes, refusals before any CUDA call,
the reference's gradients against differences, and the derived gradient formulas (CPU only)."""
import glob
import os
import re

import pytest

torch = pytest.importorskip("torch")

import moe_ref as R  # noqa: E402
from megatron_tensor_mlp_gb300 import build as B  # noqa: E402

B.build()
from megatron_tensor_mlp_gb300 import tpmlp as T  # noqa: E402

MB = 0x1000000
REACHED = (T.OK, T.ERR_CUDA, T.ERR_ARCH)


def addr(i):
    """16-byte aligned addresses 16 MB apart that are never dereferenced."""
    return 0x7F0000000000 + i * MB


def test_workspaces():
    assert T.tpmlp_layernorm_ws_bytes(4, 64) == 4 * 2 * 64 * 4
    assert T.tpmlp_layernorm_ws_bytes(1 << 20, 64) == T.tpmlp_layernorm_ws_bytes(1 << 21, 64)
    assert T.tpmlp_layernorm_ws_bytes(0, 64) == 0
    assert T.tpmlp_layernorm_ws_bytes(4, 16385) == -1 and T.tpmlp_layernorm_ws_bytes(-1, 64) == -1 and T.tpmlp_layernorm_ws_bytes(4, 0) == -1
    assert T.tpmlp_moe_route_ws_bytes(100, 64, 2) > 0 and T.tpmlp_moe_route_ws_bytes(0, 64, 2) == 0
    assert T.tpmlp_moe_route_ws_bytes(100, 1025, 2) == -1 and T.tpmlp_moe_route_ws_bytes(100, 64, 33) == -1
    assert T.tpmlp_moe_route_ws_bytes(100, 4, 5) == -1


def norm_fwd(**kw):
    a = dict(X=addr(0), gamma=addr(1), beta=addr(2), Y=addr(3), mean=addr(4), rstd=addr(5), rows=16, h=64, ldx=64, ldy=64, eps=1e-5,
             dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_layernorm_fwd(**a, check=False)


def norm_bwd(**kw):
    a = dict(X=addr(0), gamma=addr(1), mean=addr(2), rstd=addr(3), dY=addr(4), dX=addr(5), dgamma=addr(6), dbeta=addr(7), ws=addr(8),
             rows=16, h=64, ldx=64, lddy=64, lddx=64, dt=T.BF16, grad_dt=T.F32, stream=0)
    a.update(kw)
    return T.tpmlp_layernorm_bwd(**a, check=False)


def test_layernorm_refusals():
    assert norm_fwd(X=None) == T.ERR_NULL and norm_fwd(Y=None) == T.ERR_NULL
    assert norm_fwd(mean=None) == T.ERR_NULL and norm_fwd(rstd=None) == T.ERR_NULL  # half a pair
    assert norm_fwd(rows=-1) == T.ERR_SHAPE and norm_fwd(h=0) == T.ERR_SHAPE and norm_fwd(h=16385, ldx=16385, ldy=16385) == T.ERR_SHAPE
    assert norm_fwd(ldx=63) == T.ERR_SHAPE and norm_fwd(ldy=63) == T.ERR_SHAPE
    assert norm_fwd(rows=1 << 30, ldx=1 << 20) == T.ERR_SHAPE
    assert norm_fwd(eps=-1.0) == T.ERR_SHAPE and norm_fwd(eps=float("nan")) == T.ERR_SHAPE and norm_fwd(eps=float("inf")) == T.ERR_SHAPE
    assert norm_fwd(dt=4) == T.ERR_DTYPE
    assert norm_fwd(X=addr(0) + 1) == T.ERR_ALIGNMENT and norm_fwd(mean=addr(4) + 2) == T.ERR_ALIGNMENT
    assert norm_fwd(X=addr(0) + 2, dt=T.F32) == T.ERR_ALIGNMENT
    assert norm_fwd(Y=addr(0)) == T.ERR_ALIAS and norm_fwd(mean=addr(3) + 4) == T.ERR_ALIAS and norm_fwd(rstd=addr(1)) == T.ERR_ALIAS
    for ok in (dict(), dict(X=addr(0) + 2), dict(gamma=None, beta=None, mean=None, rstd=None), dict(h=63)):
        assert norm_fwd(**ok) in REACHED
    assert norm_bwd(mean=None) == T.ERR_NULL and norm_bwd(ws=None) == T.ERR_NULL and norm_bwd(dX=None) == T.ERR_NULL
    assert norm_bwd(lddx=63) == T.ERR_SHAPE and norm_bwd(h=20000, ldx=20000, lddy=20000, lddx=20000) == T.ERR_SHAPE
    assert norm_bwd(grad_dt=7) == T.ERR_DTYPE and norm_bwd(dt=7) == T.ERR_DTYPE
    assert norm_bwd(dgamma=addr(6) + 2) == T.ERR_ALIGNMENT and norm_bwd(ws=addr(8) + 8) == T.ERR_ALIGNMENT
    assert norm_bwd(dX=addr(4)) == T.ERR_ALIAS and norm_bwd(ws=addr(6) + 16) == T.ERR_ALIAS and norm_bwd(dbeta=addr(6)) == T.ERR_ALIAS
    for ok in (dict(), dict(dgamma=None), dict(dgamma=None, dbeta=None, ws=None), dict(gamma=None), dict(dgamma=addr(6) + 2, grad_dt=T.BF16)):
        assert norm_bwd(**ok) in REACHED


def route(**kw):
    a = dict(logits=addr(0), ids=addr(1), weights=addr(2), offsets=addr(3), row_token=addr(4), slot_row=addr(5), ws=addr(6), tokens=16,
             experts=8, k=2, chosen=1, dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_moe_route(**a, check=False)


def route_bwd(**kw):
    a = dict(logits=addr(0), ids=addr(1), weights=addr(2), dweights=addr(3), dlogits=addr(4), tokens=16, experts=8, k=2, chosen=1,
             dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_moe_route_bwd(**a, check=False)


def test_route_refusals():
    for name in ("logits", "ids", "weights", "offsets", "row_token", "slot_row", "ws"):
        assert route(**{name: None}) == T.ERR_NULL
    assert route(offsets=None, tokens=0) == T.ERR_NULL
    assert route(tokens=-1) == T.ERR_SHAPE and route(experts=0) == T.ERR_SHAPE and route(experts=1025) == T.ERR_SHAPE
    assert route(k=0) == T.ERR_SHAPE and route(k=9) == T.ERR_SHAPE and route(k=33, experts=64) == T.ERR_SHAPE
    assert route(tokens=1 << 27) == T.ERR_SHAPE and route(tokens=1 << 25) == T.ERR_SHAPE
    assert route(dt=2) == T.ERR_DTYPE
    assert route(ids=addr(1) + 2) == T.ERR_ALIGNMENT and route(logits=addr(0) + 1) == T.ERR_ALIGNMENT
    assert route(ws=addr(6) + 4) == T.ERR_ALIGNMENT
    assert route(ids=addr(0)) == T.ERR_ALIAS and route(slot_row=addr(4)) == T.ERR_ALIAS
    assert route() in REACHED
    for name in ("logits", "ids", "weights", "dweights", "dlogits"):
        assert route_bwd(**{name: None}) == T.ERR_NULL
    assert route_bwd(k=0) == T.ERR_SHAPE and route_bwd(dt=5) == T.ERR_DTYPE
    assert route_bwd(dlogits=addr(0)) == T.ERR_ALIAS and route_bwd(dweights=addr(3) + 1) == T.ERR_ALIGNMENT
    assert route_bwd() in REACHED


def matmul(**kw):
    a = dict(X=addr(0), row_token=addr(1), offsets=addr(2), W=addr(3), bias=None, Y=addr(4), H=None, tokens=8, rows=16, experts=4, K=64,
             N=256, act=T.ACT_NONE, out_dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_moe_matmul(**a, check=False)


def dx(**kw):
    a = dict(dY=addr(0), offsets=addr(1), W=addr(2), H=None, dX=addr(3), rows=16, experts=4, K=128, N=64, act=T.ACT_NONE, dx_dt=T.BF16,
             stream=0)
    a.update(kw)
    return T.tpmlp_moe_matmul_dx(**a, check=False)


def dw(**kw):
    a = dict(X=addr(0), row_token=addr(1), offsets=addr(2), dY=addr(3), dW=addr(4), dbias=addr(5), tokens=8, rows=16, experts=4, K=64,
             N=128, grad_dt=T.F32, stream=0)
    a.update(kw)
    return T.tpmlp_moe_matmul_dw(**a, check=False)


def test_product_refusals():
    for f, names in ((matmul, ("X", "offsets", "W", "Y")), (dx, ("dY", "offsets", "W", "dX")), (dw, ("X", "offsets", "dY", "dW"))):
        for name in names:
            assert f(**{name: None}) == T.ERR_NULL, name
        assert f(rows=-1) == T.ERR_SHAPE and f(experts=0) == T.ERR_SHAPE and f(experts=1025) == T.ERR_SHAPE
        assert f(K=0) == T.ERR_SHAPE and f(N=0) == T.ERR_SHAPE and f(K=1 << 30, N=1 << 14) == T.ERR_SHAPE
        assert f(K=68) == T.ERR_ALIGNMENT and f(N=68) == T.ERR_ALIGNMENT and f(offsets=addr(1) + 2) == T.ERR_ALIGNMENT
        assert f() in REACHED
    for f in (matmul, dw):
        assert f(row_token=None) == T.ERR_SHAPE  # X then has the rows themselves
        assert f(row_token=None, tokens=16) in REACHED
        assert f(tokens=0) == T.ERR_SHAPE and f(tokens=-1) == T.ERR_SHAPE
        assert f(X=addr(0) + 8) == T.ERR_ALIGNMENT and f(row_token=addr(1) + 2) == T.ERR_ALIGNMENT
    assert matmul(H=addr(5)) == T.ERR_SHAPE  # (of the gated activation only)
    assert matmul(act=T.ACT_GELU_ERF) == T.ERR_SHAPE and matmul(act=9) == T.ERR_SHAPE
    assert matmul(act=T.ACT_SWIGLU, N=384) == T.ERR_DIVISIBILITY
    assert matmul(act=T.ACT_SWIGLU, out_dt=T.F32) == T.ERR_DTYPE and matmul(out_dt=5) == T.ERR_DTYPE
    assert matmul(Y=addr(0)) == T.ERR_ALIAS and matmul(act=T.ACT_SWIGLU, H=addr(4) + 16) == T.ERR_ALIAS
    assert matmul(act=T.ACT_SWIGLU, H=addr(5), bias=addr(6)) in REACHED
    assert dx(act=T.ACT_SWIGLU) == T.ERR_NULL  # without H
    assert dx(H=addr(4)) == T.ERR_SHAPE
    assert dx(act=T.ACT_SWIGLU, H=addr(4), K=192) == T.ERR_DIVISIBILITY
    assert dx(act=T.ACT_SWIGLU, H=addr(4), dx_dt=T.F32) == T.ERR_DTYPE
    assert dx(act=T.ACT_SWIGLU, H=addr(3)) == T.ERR_ALIAS and dx(dX=addr(2)) == T.ERR_ALIAS
    assert dx(act=T.ACT_SWIGLU, H=addr(4)) in REACHED and dx(dx_dt=T.F32) in REACHED
    assert dw(grad_dt=3) == T.ERR_DTYPE and dw(dbias=addr(4)) == T.ERR_ALIAS and dw(dW=addr(0)) == T.ERR_ALIAS
    assert dw(dbias=None, grad_dt=T.BF16) in REACHED


def combine(**kw):
    a = dict(O=addr(0), slot_row=addr(1), weights=addr(2), Z=addr(3), tokens=8, rows=16, k=2, h=64, stream=0)
    a.update(kw)
    return T.tpmlp_moe_combine(**a, check=False)


def combine_bwd(**kw):
    a = dict(O=addr(0), slot_row=addr(1), weights=addr(2), dZ=addr(3), dO=addr(4), dweights=addr(5), tokens=8, rows=16, k=2, h=64, stream=0)
    a.update(kw)
    return T.tpmlp_moe_combine_bwd(**a, check=False)


def test_combine_refusals():
    assert combine(O=None) == T.ERR_NULL and combine(slot_row=None) == T.ERR_NULL and combine(Z=None) == T.ERR_NULL
    assert combine(k=0) == T.ERR_SHAPE and combine(k=33) == T.ERR_SHAPE and combine(h=0) == T.ERR_SHAPE and combine(rows=-1) == T.ERR_SHAPE
    assert combine(h=68) == T.ERR_ALIGNMENT and combine(Z=addr(3) + 8) == T.ERR_ALIGNMENT and combine(weights=addr(2) + 2) == T.ERR_ALIGNMENT
    assert combine(Z=addr(0)) == T.ERR_ALIAS and combine(Z=addr(2)) == T.ERR_ALIAS
    assert combine() in REACHED and combine(weights=None) in REACHED and combine(O=None, rows=0) in REACHED
    assert combine_bwd(O=None) == T.ERR_NULL and combine_bwd(dO=None) == T.ERR_NULL and combine_bwd(dZ=None) == T.ERR_NULL
    assert combine_bwd(dO=addr(3)) == T.ERR_ALIAS and combine_bwd(dweights=addr(4)) == T.ERR_ALIAS
    assert combine_bwd(O=None, dweights=None) in REACHED and combine_bwd() in REACHED


def test_act_of_the_other_layers_is_unchanged():
    """The gated activation belongs to the grouped products: the column layer refuses it as before."""
    st = T.tpmlp_column_fwd(addr(0), addr(1), None, addr(2), None, 4, 2, 64, 256, 2, act=T.ACT_SWIGLU, stream=0, check=False)
    assert st == T.tpmlp_column_fwd(addr(0), addr(1), None, addr(2), None, 4, 2, 64, 256, 2, act=9, stream=0, check=False) != T.OK


def test_calls_of_nothing_pass_without_pointers():
    for st in (T.tpmlp_layernorm_fwd(None, None, None, None, None, None, 0, 64, 64, 64, stream=0, check=False),
               T.tpmlp_moe_route_bwd(None, None, None, None, None, 0, 8, 2, stream=0, check=False),
               T.tpmlp_moe_matmul(None, None, addr(0), addr(1), None, None, None, 0, 0, 4, 64, 64, stream=0, check=False),
               T.tpmlp_moe_matmul_dx(None, addr(0), addr(1), None, None, 0, 4, 64, 64, stream=0, check=False),
               T.tpmlp_moe_combine(None, None, None, None, 0, 0, 2, 64, stream=0, check=False)):
        assert st in REACHED


# ------------------------------------------------------------------ formulas against differences, in 64 bits
def differences(f, x, step=1e-6):
    """The gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        hi = float(f())
        flat[i] = keep - step
        lo = float(f())
        flat[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return g


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, dtype=R.D)  # noqa: E731
    x, gamma, beta, dy = n(3, 10), n(10), n(10), n(3, 10)
    f = lambda: (R.norm(x, gamma, beta, 1e-5)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = R.norm(x, gamma, beta, 1e-5)
    for got, v in zip(R.norm_bwd(x, gamma, mean, rstd, dy), (x, gamma, beta)):
        assert torch.allclose(got, differences(f, v), atol=1e-7)


@pytest.mark.parametrize("chosen", [0, 1])
def test_route_gradient_against_differences(chosen):
    g = torch.Generator().manual_seed(1)
    x, dw = torch.randn(4, 6, generator=g, dtype=R.D), torch.randn(4, 3, generator=g, dtype=R.D)
    f = lambda: (R.route(x, 3, chosen)[1] * dw).sum()  # noqa: E731
    ids, w = R.route(x, 3, chosen)[:2]
    ref = R.route_bwd(x, ids, dw, chosen)
    assert torch.allclose(ref, differences(f, x), atol=1e-7)
    # the kernel's formula
    p = torch.zeros_like(x).scatter(1, ids.long(), w) if chosen else torch.softmax(x, 1)
    d = torch.zeros_like(x).scatter(1, ids.long(), dw)
    assert torch.allclose(p * (d - (w * dw).sum(1, keepdim=True)), ref, atol=1e-12)


def test_gated_expert_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, dtype=R.D)  # noqa: E731
    off = torch.tensor([0, 2, 2, 3])
    x, w1, w2, do = n(3, 2), n(3, 2, 256), n(3, 128, 2), n(3, 2)

    def f():
        gate, up = R.halves(R.matmul(x, off, w1)[0])
        return (R.matmul(R.silu(gate) * up, off, w2)[0] * do).sum()

    h = R.matmul(x, off, w1)[0]
    gate, up = R.halves(h)
    d = R.matmul(do, off, w2.transpose(1, 2))[0]
    dh = R.packed(d * up * R.dsilu(gate), d * R.silu(gate))
    assert torch.allclose(R.matmul(dh, off, w1.transpose(1, 2))[0], differences(f, x), atol=1e-6)
    assert torch.allclose(R.dw(x, off, dh, 3)[0], differences(f, w1), atol=1e-6)
    assert torch.allclose(R.dw(R.silu(gate) * up, off, do, 3)[0], differences(f, w2), atol=1e-6)


# ------------------------------------------------------------------ sources
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "megatron_tensor_mlp_gb300", "csrc")
SOURCES = sorted(os.path.basename(f) for pat in ("moe*.cu*", "layernorm.cu") for f in glob.glob(os.path.join(CSRC, pat)))


@pytest.mark.parametrize("name", SOURCES)
def test_no_non_coherent_load_behind_the_wait(name):
    """These kernels start while the kernel ahead in the stream still runs and read what it writes: a non-coherent load
    asks for memory that nobody writes while the kernel is resident."""
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    found = re.findall(r"__ldg|__restrict__|ld\.global(?:\.\w+)*\.nc", code)
    assert not found, found


def test_an_expert_s_tiles_are_never_empty():
    """tile_tokens: ceil(n / TN) tiles of equal size, a multiple of 16, cover an expert's rows and leave none empty."""
    for tn in (128, 256):
        for n in range(1, 20 * tn):
            nt = -(-n // tn)
            size = (-(-n // nt) + 15) // 16 * 16
            assert size <= tn and (nt - 1) * size < n <= nt * size, (tn, n)


def test_a_layer_on_the_cpu_is_refused():
    """Its calls would hand over addresses that the GPU cannot read."""
    from megatron_tensor_mlp_gb300.moe_block import ExpertLayer
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        ExpertLayer(z(8), z(8), z(8, 8), z(8, 8, 128), z(8, 8, 128), z(8, 128, 8), 2)
