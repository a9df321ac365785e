"""MXFP4 operators where the ordinary tests do not reach: the single-CTA kernels with three CTAs an SM, K loops of
hundreds of thousands, and weight gradients over a long token axis."""
import numpy as np
import pytest

import gpu_util as U
import mxfp4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import tpmlp
    return tpmlp


@pytest.fixture
def set_mode(T):
    yield T.tpmlp_set_mxfp4_mode
    T.tpmlp_set_mxfp4_mode(0)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def normal(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def operand(T, x):
    """x [rows, k] bf16 on the device -> (codes, scales) with NaN scales where no product may look, and the values."""
    o = T.mxfp4_empty(*x.shape)
    o[1].fill_(255)
    T.tpmlp_mxfp4_quantize(x, *o, None, None, *x.shape, x.shape[1])
    return o, R.q(host(x))


def many_tiles():
    """Column tiles of 128 that are more than two CTAs for every SM: few rows then take three CTAs an SM."""
    import torch
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count + 9


@pytest.mark.parametrize("k", [32, 136, 1312])
@pytest.mark.parametrize("m", [1, 16, 17, 32])
def test_product_of_few_rows_and_many_tiles(T, m, k):
    """Rings of three stages, walked once at most and many times over; the last tile is ragged."""
    import torch
    n = many_tiles() * 128 - 56
    (aq, as_), a = operand(T, normal(m, m, k))
    (bq, bs), b = operand(T, normal(k, n, k))
    bias = normal(3, n)
    for out_dt, tdt, with_bias in ((T.BF16, torch.bfloat16, True), (T.F32, torch.float32, False)):
        D = torch.full((m + 1, n), 7.0, dtype=tdt, device="cuda")
        T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, bias if with_bias else None, D, m, n, k, out_dt)
        T.tpmlp_device_status()
        assert bool((D[m] == 7.0).all()), "written past the last row"
        R.assert_product(host(D[:m]), a, b, host(bias) if with_bias else None, out_dt == T.BF16, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,h", [(1, 1032), (5, 256), (32, 264)])
def test_forward_of_few_tokens_and_many_features(T, m, h):
    import torch
    f = (many_tiles() + 1) // 2 * 128
    X, W, B = normal(1, m, h), normal(2, h, 2 * f, scale=h ** -0.5), normal(3, f, h, scale=f ** -0.5)
    bw, b2 = normal(4, 2 * f, scale=0.1), normal(5, h, scale=0.1)
    Wt, Bt = T.mxfp4_empty(2 * f, h), T.mxfp4_empty(h, f)
    T.tpmlp_mxfp4_quantize(W, None, None, *Wt, h, 2 * f, 2 * f)
    T.tpmlp_mxfp4_quantize(B, None, None, *Bt, f, h, h)
    n = T.tpmlp_mxfp4_swiglu_ws_bytes(m, 1, h, f, 1, 0)
    for bias in (False, True):
        ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        Z, H = (torch.full((m + 1, c), 7.0, dtype=torch.bfloat16, device="cuda") for c in (h, 2 * f))
        Z2 = torch.empty((m, h), dtype=torch.bfloat16, device="cuda")
        args = (X, *Wt, bw if bias else None, *Bt, b2 if bias else None)
        T.tpmlp_mxfp4_swiglu_mlp_fwd(*args, Z, H, ws, m, 1, h, f, 1)
        T.tpmlp_mxfp4_swiglu_mlp_fwd(*args, Z2, None, ws, m, 1, h, f, 1)
        T.tpmlp_device_status()
        assert bool((Z[m] == 7.0).all()) and bool((H[m] == 7.0).all()) and bool((ws[n:] == 0xFF).all())
        assert torch.equal(Z[:m], Z2)
        Zr, Hr = R.block_fwd(host(X), R.q(host(W).T), R.q(host(B).T), host(bw) if bias else None, host(b2) if bias else None)
        U.assert_close(host(H[:m]), Hr, "bf16", "H")
        U.assert_close(host(Z[:m]), Zr, "bf16", "Z")


@pytest.mark.parametrize("mode", [0, 1, 2, 5], ids=["auto", "single", "pair", "split8"])
@pytest.mark.parametrize("m,n,k", [(1, 128, 20480), (150, 272, 5120), (150, 272, 20480), (300, 264, 65536)])
def test_fp32_product_keeps_its_bits(T, set_mode, mode, m, n, k):
    """fp32 D at a rank's K against 64 bits in the Frobenius norm, beside the elementwise bound, whose sum of magnitudes
    leaves room for a result rounded to fewer bits.  Each 64-deep step of the tensor cores and each partial sum of a split
    moves a value by at most 2^-23 of its partial sum, and with operands of either sign the partial sums' norm stays below
    the result's: (K / 64 + 16) 2^-23 of it, 4e-5 at K = 20480 (a value rounded to bf16 is off by 1.7e-3, to 16
    bits by 7e-6 a step)."""
    import torch
    set_mode(mode)
    (aq, as_), a = operand(T, normal(m, m, k))
    (bq, bs), b = operand(T, normal(n + 1, n, k))
    D = torch.empty((m, n), device="cuda")
    T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
    T.tpmlp_device_status()
    ref = a @ b.T
    off = np.linalg.norm(host(D) - ref) / np.linalg.norm(ref)
    assert off <= (-(-k // 64) + 16) * 2.0 ** -23, off
    R.assert_product(host(D), a, b, None, False)


@pytest.mark.parametrize("mode", [0, 1, 2], ids=["auto", "single", "pair"])
def test_product_of_a_very_long_axis(T, set_mode, mode):
    """K of 262144 and a ragged end, with operands of one sign: every partial sum's rounding goes the same way if the
    tensor cores cut it off, and shows against the bound of one unit for each step."""
    import torch
    set_mode(mode)
    m, n, k = 40, 136, 262144 + 96
    (aq, as_), a = operand(T, normal(1, m, k).abs())
    (bq, bs), b = operand(T, normal(2, n, k).abs())
    D = torch.empty((m, n), device="cuda")
    T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
    T.tpmlp_device_status()
    R.assert_product(host(D), a, b, None, False, "one sign")


def test_weight_gradients_over_many_tokens(T):
    """215001 tokens: the codes along the tokens and along the features pass 2^32 bytes.  Columns of dW, rows of dB and
    bias gradients from either end of the features against 64 bits over all tokens."""
    import torch
    m, h, f = 215_001, 64, 20480
    X, dZ = normal(1, m, h), normal(2, m, h)
    W, B = normal(3, h, 2 * f, scale=h ** -0.5), normal(4, f, h, scale=f ** -0.5)
    H = torch.empty((m, 2 * f), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    Wn, Bn = T.mxfp4_empty(h, 2 * f), T.mxfp4_empty(f, h)
    T.tpmlp_mxfp4_quantize(W, *Wn, None, None, h, 2 * f, 2 * f)
    T.tpmlp_mxfp4_quantize(B, *Bn, None, None, f, h, h)
    dX, dW, dB = torch.empty((m, h), device="cuda"), torch.empty((h, 2 * f), device="cuda"), torch.empty((f, h), device="cuda")
    dbw, db2 = torch.empty(2 * f, device="cuda"), torch.empty(h, device="cuda")
    ws = torch.full((T.tpmlp_mxfp4_swiglu_ws_bytes(m, 1, h, f, 1, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    T.tpmlp_mxfp4_swiglu_mlp_bwd(X, *Wn, *Bn, H, dZ, dX, dW, dB, dbw, db2, ws, m, 1, h, f, 1, dx_dt=T.F32)
    T.tpmlp_device_status()
    del ws
    pick = np.r_[0:16, f // 2:f // 2 + 16, f - 16:f]  # features
    gate = pick // 128 * 256 + pick % 128             # their columns of H and dW; up 128 further
    g, u = host(H[:, gate]), host(H[:, gate + 128])
    x, dz = host(X), host(dZ)
    s = R.sigmoid(g)
    dy = R.q(dz) @ R.q(host(B[pick])).T
    dg, du, y = dy * u * s * (1 + g * (1 - s)), dy * g * s, g * s * u
    xt = R.q(x.T)
    for name, cols, d in (("gate", gate, dg), ("up", gate + 128, du)):
        U.assert_close(host(dW[:, cols]), xt @ R.q(d.T).T, "bf16", f"dW {name}")
        U.assert_close(host(dbw[cols]), d.sum(0), "bf16", f"dbw {name}")
    U.assert_close(host(dB[pick]), R.q(y.T) @ R.q(dz.T).T, "bf16", "dB")
    U.assert_close(host(db2), dz.sum(0), "bf16", "db2")
    # dX: the last tokens over all features
    t = slice(m - 40, m)
    ref = R.block_bwd(x[t], R.q(host(W)), R.q(host(B)), host(H[t]), dz[t])[0]
    U.assert_close(host(dX[t]), ref, "bf16", "dX")


@pytest.mark.parametrize("mode", [0, 1, 2, 4], ids=["auto", "single", "pair", "split4"])
@pytest.mark.parametrize("k", [5120, 20480, 262144 + 96])
@pytest.mark.parametrize("one_sign", [False, True], ids=["signs", "one-sign"])
def test_products_of_blocks_of_many_sizes(T, set_mode, mode, k, one_sign):
    """Blocks of 2^-16 to 1 times the same values: with blocks of one size nearly every partial sum is a number of 24 bits,
    here they have to be rounded.  The bounds are those above."""
    import torch
    set_mode(mode)
    m, n = 40, 136

    def blocks(seed, rows):
        x = normal(seed, rows, k)
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        e = torch.randint(-16, 1, (rows, -(-k // 32)), generator=g, device="cuda").repeat_interleave(32, dim=1)[:, :k]
        x = torch.ldexp(x.float(), e).to(torch.bfloat16)
        return x.abs() if one_sign else x

    (aq, as_), a = operand(T, blocks(1, m))
    (bq, bs), b = operand(T, blocks(2, n))
    D = torch.empty((m, n), device="cuda")
    T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
    T.tpmlp_device_status()
    ref = a @ b.T
    off = np.linalg.norm(host(D) - ref) / np.linalg.norm(ref)
    assert off <= (-(-k // 64) + 16) * 2.0 ** -23, off
    R.assert_product(host(D), a, b, None, False)
