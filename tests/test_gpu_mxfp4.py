"""MXFP4 operators on the GPU against 64-bit references (mxfp4_ref): the quantiser bit for bit, the
product within its derived bound in every tiling, the gated block's forward and backward."""
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


@pytest.fixture(params=[0, 1, 2, 3, 4, 5], ids=["auto", "single", "pair", "split2", "split4", "split8"])
def mode(request, T):
    T.tpmlp_set_mxfp4_mode(request.param)
    yield request.param
    T.tpmlp_set_mxfp4_mode(0)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def operand(T, x):
    """Values [rows, k] quantised by the reference -> device (codes, tiled scales) and the exact values."""
    import torch
    codes, scales = R.quantize(x)
    # scale bytes of rows past the last are not used: NaN there must not show
    t = R.tile_scales(scales, x.shape[0], x.shape[1], fill=255)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(t).cuda(), R.dequantize(codes, scales, x.shape[1])


def wild(rng, rows, cols, f32):
    """Values over many magnitudes with ties, zeros, saturating and tiny blocks."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, cols)))
    x[rng.random((rows, cols)) < 0.2] *= 0.0
    grid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9], (rows, cols)) * rng.choice([-1, 1], (rows, cols))
    pick = rng.random(rows) < 0.4
    x[pick] = grid[pick] * np.exp2(rng.integers(-140, 120, (rows, 1)))[pick]
    x[rng.random(rows) < 0.05] = 0.0
    with np.errstate(over="ignore"):
        x = x.astype(np.float32)
    if not f32:
        x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    return x


def to_device(x, f32):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if f32 else t.to(torch.bfloat16)


def check_operand(codes, scales, x, what):
    """Device codes and scales against the reference's for x [rows, k]."""
    want, sc = R.quantize(x)
    assert np.array_equal(codes.cpu().numpy(), want), f"{what}: codes differ"
    got = R.untile_scales(scales.cpu().numpy(), x.shape[0], x.shape[1])
    assert np.array_equal(got[:, : sc.shape[1]], sc), f"{what}: scales differ"
    assert not got[:, sc.shape[1]:].any(), f"{what}: a padding block's scale is not zero"


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 5120), (3, 8), (5, 40), (31, 64), (33, 96), (127, 136), (128, 128), (129, 256),
                                       (150, 272), (300, 520), (257, 1000)])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_quantize_bit_exact(T, rows, cols, f32):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = wild(rng, rows, cols, f32)
    t, dt = to_device(x, f32), T.F32 if f32 else T.BF16
    for along, across in ((True, False), (False, True), (True, True)):
        a, b = T.mxfp4_empty(rows, cols), T.mxfp4_empty(cols, rows)
        for o in a + b:
            o.fill_(0xAA)
        T.tpmlp_mxfp4_quantize(t, *(a if along else (None, None)), *(b if across else (None, None)), rows, cols, cols, 1, dt)
        T.tpmlp_device_status()
        if along:
            check_operand(*a, x, "along the columns")
        if across:
            check_operand(*b, x.T, "along the rows")
        for o in (() if along else a) + (() if across else b):
            assert bool((o == 0xAA).all())


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_quantize_ragged_columns_of_a_wider_matrix(T, f32):
    """A column slice whose width is no multiple of 8, at an offset, row pitch wider than the slice; what lies
    beside it (NaN) is not looked at."""
    rng = np.random.default_rng(5)
    for rows, cols, ldx, off in [(70, 37, 64, 8), (130, 1, 16, 0), (9, 131, 160, 24)]:
        x = np.full((rows, ldx), np.nan, dtype=np.float32)
        x[:, off:off + cols] = wild(rng, rows, cols, f32)
        t = to_device(x, f32)
        a, b = T.mxfp4_empty(rows, cols), T.mxfp4_empty(cols, rows)
        T.tpmlp_mxfp4_quantize(t[:, off:], *a, *b, rows, cols, ldx, 1, T.F32 if f32 else T.BF16)
        a2 = T.mxfp4_empty(rows, cols)
        T.tpmlp_mxfp4_quantize(t[:, off:], *a2, None, None, rows, cols, ldx, 1, T.F32 if f32 else T.BF16)
        T.tpmlp_device_status()
        v = x[:, off:off + cols]
        check_operand(*a, v, "along the columns")
        check_operand(*a2, v, "along the columns only")
        check_operand(*b, v.T, "along the rows")


@pytest.mark.parametrize("rows,cols,p", [(40, 256, 2), (129, 384, 3), (64, 256, 8)])
def test_quantize_column_shards(T, rows, cols, p):
    """Column shards [p][rows][cols/p] give the operands of the unsharded matrix."""
    x = wild(np.random.default_rng(p), rows, cols, False)
    t = to_device(x, False).view(rows, p, cols // p).transpose(0, 1).contiguous()
    a, b = T.mxfp4_empty(rows, cols), T.mxfp4_empty(cols, rows)
    T.tpmlp_mxfp4_quantize(t, *a, *b, rows, cols, cols // p, p)
    a2 = T.mxfp4_empty(rows, cols)
    T.tpmlp_mxfp4_quantize(t, *a2, None, None, rows, cols, cols // p, p)
    T.tpmlp_device_status()
    check_operand(*a, x, "along the columns")
    check_operand(*a2, x, "along the columns only")
    check_operand(*b, x.T, "along the rows")


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_quantize_not_finite_and_extremes(T, f32):
    """A NaN or an infinity makes its block the NaN scale with zero codes, and no other block; the largest and
    the smallest numbers of the type."""
    x = np.ones((64, 96), dtype=np.float32)
    x[3, 40], x[7, 0], x[9, 95], x[40, 5] = np.nan, np.inf, -np.inf, np.nan
    x[5, :32] = 0.0
    x[6, :32] = -0.0
    big = np.float32(3.3895314e38)  # the largest bf16
    x[11, :32] = big
    x[12, 32:64] = -big
    x[13, :32] = np.float32(2.0 ** -133)  # subnormal
    x[14, :32] = np.float32(2.0 ** -126)
    x[15, :32] = np.float32(2.0 ** -125)
    if f32:
        x[16, :32] = np.float32(1e-45)
    t = to_device(x, f32)
    a, b = T.mxfp4_empty(64, 96), T.mxfp4_empty(96, 64)
    T.tpmlp_mxfp4_quantize(t, *a, *b, 64, 96, 96, 1, T.F32 if f32 else T.BF16)
    check_operand(*a, x, "along the columns")
    check_operand(*b, x.T, "along the rows")
    import torch
    for dt, tdt in ((T.F32, torch.float32), (T.BF16, torch.bfloat16)):
        out = torch.empty((64, 96), dtype=tdt, device="cuda")
        T.tpmlp_mxfp4_dequantize(*a, out, 64, 96, dt)
        T.tpmlp_device_status()
        assert np.array_equal(host(out), R.dequantize(*R.quantize(x), 96), equal_nan=True)


@pytest.mark.parametrize("rows,k", [(1, 1), (3, 37), (130, 264), (5, 12)])
def test_dequantize(T, rows, k):
    import torch
    codes, scales, v = operand(T, wild(np.random.default_rng(k), rows, k, True))
    for dt, tdt in ((T.F32, torch.float32), (T.BF16, torch.bfloat16)):
        out = torch.full((rows * k + 8,), 7.0, dtype=tdt, device="cuda")
        T.tpmlp_mxfp4_dequantize(codes, scales, out, rows, k, dt)
        T.tpmlp_device_status()
        assert np.array_equal(host(out)[: rows * k].reshape(rows, k), v)
        assert bool((out[rows * k:] == 7.0).all())


SHAPES = [(1, 8, 32), (1, 128, 1024), (16, 136, 2048), (17, 256, 2080), (33, 64, 96), (65, 392, 512), (128, 128, 256), (129, 264, 1056),
          (150, 272, 136), (256, 256, 64), (257, 520, 320), (400, 1032, 5120)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(T, m, n, k, mode):
    import torch
    rng = np.random.default_rng(m + n + k)
    scale = np.exp2(rng.integers(-3, 4, (m, 1)))
    aq, as_, a = operand(T, rng.standard_normal((m, k)) * scale)
    bq, bs, b = operand(T, rng.standard_normal((n, k)))
    bias = rng.standard_normal(n).astype(np.float32)
    bias_d = bf16(bias)
    for out_dt, tdt, with_bias in ((T.BF16, torch.bfloat16, True), (T.F32, torch.float32, False), (T.F32, torch.float32, True)):
        D = torch.full((m + 1, n), 7.0, dtype=tdt, device="cuda")
        T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, bias_d if with_bias else None, D, m, n, k, out_dt)
        T.tpmlp_device_status()
        assert bool((D[m] == 7.0).all()), "written past the last row"
        R.assert_product(host(D[:m]), a, b, host(bias_d) if with_bias else None, out_dt == T.BF16, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 4, 1), (7, 16, 1), (20, 24, 33), (5, 12, 40), (130, 260, 31)])
def test_product_smallest_and_odd(T, m, n, k, mode):
    """One value of k, K that ends inside a block, rows of fp32 D that are no multiple of 8 long."""
    import torch
    rng = np.random.default_rng(m * n + k)
    aq, as_, a = operand(T, rng.standard_normal((m, k)))
    bq, bs, b = operand(T, rng.standard_normal((n, k)))
    bias = bf16(rng.standard_normal(n))
    for out_dt, tdt in ((T.F32, torch.float32),) + (((T.BF16, torch.bfloat16),) if n % 8 == 0 else ()):
        D = torch.full((m + 1, n), 7.0, dtype=tdt, device="cuda")
        T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, bias, D, m, n, k, out_dt)
        T.tpmlp_device_status()
        assert bool((D[m] == 7.0).all())
        R.assert_product(host(D[:m]), a, b, host(bias), out_dt == T.BF16, f"{m}x{n}x{k}")


def test_block_not_finite_rows(T):
    """A NaN in one token's input makes that token's output NaN and no other's; extreme gates (the sigmoid at 0 and 1)
    stay finite."""
    import torch
    s, b, h, f, p = 70, 1, 256, 512, 1
    d = make_block(T, s, b, h, f, p, seed=40)
    X = d["X"].clone()
    X[5, 17] = float("nan")
    bw = d["bw"].clone()
    bw[:64], bw[64:128] = 3e4, -3e4
    Z, H = torch.empty_like(X), torch.empty((s, 2 * f), dtype=torch.bfloat16, device="cuda")
    ws, _ = workspace(T, s, b, h, f, p, 0)
    T.tpmlp_mxfp4_swiglu_mlp_fwd(X, *d["Wt"], bw, *d["Bt"], None, Z, H, ws, s, b, h, f, p)
    T.tpmlp_device_status()
    z = host(Z)
    rest = np.arange(s) != 5
    assert np.isnan(z[5]).all()
    Zr, Hr = R.block_fwd(host(X[torch.from_numpy(rest).cuda()]), R.q(host(d["W"]).T), R.q(host(d["B"]).T), host(bw))
    U.assert_close(z[rest], Zr, "bf16", "Z")
    U.assert_close(host(H)[rest], Hr, "bf16", "H")
    dX, dW, dB = torch.empty_like(X), torch.empty((p, h, 2 * f), device="cuda"), torch.empty((f, h), device="cuda")
    Hc = torch.where(H.isnan(), torch.zeros_like(H), H)
    ws, _ = workspace(T, s, b, h, f, p, 1)
    T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], Hc, d["dZ"], dX, dW, dB, None, None, ws, s, b, h, f, p)
    T.tpmlp_device_status()
    with np.errstate(over="ignore"):
        ref = R.block_bwd(host(d["X"]), R.q(host(d["W"])), R.q(host(d["B"])), host(Hc), host(d["dZ"]))
    U.assert_close(host(dX), ref[0], "bf16", "dX")
    U.assert_close(host(dW[0]), ref[1], "bf16", "dW")
    U.assert_close(host(dB), ref[2], "bf16", "dB")


def test_product_many_tiles_and_repeats(T):
    """Several waves of pair tiles, and the same bits twice in every tiling."""
    import torch
    m, n, k = 2100, 2568, 1312
    rng = np.random.default_rng(3)
    aq, as_, a = operand(T, rng.standard_normal((m, k)))
    bq, bs, b = operand(T, rng.standard_normal((n, k)))
    for md in (0, 1, 2, 4):
        T.tpmlp_set_mxfp4_mode(md)
        try:
            outs = []
            for _ in range(2):
                D = torch.full((m, n), float("nan"), device="cuda")
                T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
                outs.append(D)
            T.tpmlp_device_status()
        finally:
            T.tpmlp_set_mxfp4_mode(0)
        assert torch.equal(outs[0], outs[1])
        R.assert_product(host(outs[0]), a, b, None, False, f"mode {md}")


@pytest.mark.parametrize("m,n,k", [(640, 1024, 8192), (150, 2500, 8000)])
def test_product_of_long_rows_and_few_tiles(T, m, n, k):
    """K split over the CTAs of a cluster, also three ways."""
    import torch
    rng = np.random.default_rng(m)
    aq, as_, a = operand(T, rng.standard_normal((m, k)))
    bq, bs, b = operand(T, rng.standard_normal((n, k)))
    outs = []
    for _ in range(2):
        D = torch.full((m + 1, n), 7.0, device="cuda")
        T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
        T.tpmlp_device_status()
        assert bool((D[m] == 7.0).all())
        outs.append(D[:m])
    assert torch.equal(outs[0], outs[1])
    R.assert_product(host(outs[0]), a, b, None, False, "auto")


@pytest.mark.parametrize("shape", [(128, 1, 4096, 2560, 1), (100, 1, 4096, 5120, 2)], ids=lambda s: "s{}b{}h{}f{}p{}".format(*s))
def test_block_of_long_rows_and_few_tiles(T, shape):
    """The gated epilogues behind a K loop split over a cluster, also three ways, against the same without a split.
    Sums in another order move a value by some 2^-20 of its size; one in 10^5 then falls on the other side of a
    rounding boundary of the 4-bit grid, a third of its size away: norms agree to sqrt(1e-5) / 3, 0.1 %; three times that."""
    import torch
    s, b, h, f, p = shape
    M = s * b
    d = make_block(T, *shape, seed=f)
    H = torch.randn((M, 2 * f), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    new = lambda *shp: torch.full(shp, float("nan"), device="cuda")  # noqa: E731
    outs = []
    for md in (1, 0):
        Z, dX, dW, dB = new(M, h), new(M, h), new(p, h, 2 * f // p), new(f, h)
        Hs, dbw, db2 = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda"), new(2 * f), new(h)
        T.tpmlp_set_mxfp4_mode(md)
        try:
            ws, _ = workspace(T, *shape, 0)
            T.tpmlp_mxfp4_swiglu_mlp_fwd(d["X"], *d["Wt"], d["bw"], *d["Bt"], d["b2"], Z, Hs, ws, *shape, z_dt=T.F32)
            ws, _ = workspace(T, *shape, 1)
            T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, dbw, db2, ws, *shape, dx_dt=T.F32)
            T.tpmlp_device_status()
        finally:
            T.tpmlp_set_mxfp4_mode(0)
        outs.append((Z, Hs, dX, dW, dB, dbw, db2))
    for name, x, y in zip(("Z", "H", "dX", "dW", "dB", "dbw", "db2"), *outs):
        off = float((x.double() - y.double()).norm() / x.double().norm())
        assert off <= 3e-3, (name, off)


def test_product_nan_block_reaches_its_row_only(T, mode):
    import torch
    m, n, k = 40, 128, 512
    rng = np.random.default_rng(9)
    x = rng.standard_normal((m, k))
    x[5, 70] = np.inf
    aq, as_, a = operand(T, x)
    bq, bs, b = operand(T, rng.standard_normal((n, k)))
    D = torch.empty((m, n), device="cuda")
    T.tpmlp_mxfp4_matmul(aq, as_, bq, bs, None, D, m, n, k, T.F32)
    T.tpmlp_device_status()
    d = host(D)
    assert np.isnan(d[5]).all()
    rest = np.arange(m) != 5
    R.assert_product(d[rest], a[rest], b, None, False)


BLOCKS = [(1, 1, 256, 256, 1), (5, 3, 264, 512, 2), (33, 1, 512, 384, 1), (129, 1, 256, 1024, 4), (75, 4, 320, 768, 2)]


def make_block(T, s, b, h, f, p, seed):
    """bf16 tensors of the block, its weights quantised by the library for both directions."""
    import torch
    rng = np.random.default_rng(seed)
    d = {"X": bf16(rng.standard_normal((s * b, h))), "dZ": bf16(rng.standard_normal((s * b, h))),
         "W": bf16(rng.standard_normal((h, 2 * f)) * h ** -0.5), "B": bf16(rng.standard_normal((f, h)) * f ** -0.5),
         "bw": bf16(rng.standard_normal(2 * f) * 0.1), "b2": bf16(rng.standard_normal(h) * 0.1)}
    W_sh = d["W"].view(h, p, 2 * f // p).transpose(0, 1).contiguous()
    d["Wn"], d["Wt"] = T.mxfp4_empty(h, 2 * f), T.mxfp4_empty(2 * f, h)
    T.tpmlp_mxfp4_quantize(W_sh, *d["Wn"], *d["Wt"], h, 2 * f, 2 * f // p, p)
    d["Bn"], d["Bt"] = T.mxfp4_empty(f, h), T.mxfp4_empty(h, f)
    T.tpmlp_mxfp4_quantize(d["B"], *d["Bn"], *d["Bt"], f, h, h)
    torch.cuda.synchronize()
    return d


def workspace(T, s, b, h, f, p, backward):
    """A workspace with a guard behind it, filled with NaN scales."""
    import torch
    n = T.tpmlp_mxfp4_swiglu_ws_bytes(s, b, h, f, p, backward)
    return torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda"), n


@pytest.mark.parametrize("shape", BLOCKS, ids=lambda s: "s{}b{}h{}f{}p{}".format(*s))
def test_block_forward(T, shape, mode):
    import torch
    s, b, h, f, p = shape
    M = s * b
    d = make_block(T, *shape, seed=sum(shape))
    w, bb = R.q(host(d["W"]).T), R.q(host(d["B"]).T)
    for bias in (False, True):
        Z = torch.full((M + 1, h), 7.0, dtype=torch.bfloat16, device="cuda")
        H = torch.full((M + 1, 2 * f), 7.0, dtype=torch.bfloat16, device="cuda")
        ws, n = workspace(T, *shape, 0)
        args = (d["X"], *d["Wt"], d["bw"] if bias else None, *d["Bt"], d["b2"] if bias else None)
        T.tpmlp_mxfp4_swiglu_mlp_fwd(*args, Z, H, ws, *shape)
        Z32 = torch.full((M, h), float("nan"), device="cuda")
        T.tpmlp_mxfp4_swiglu_mlp_fwd(*args, Z32, None, ws, *shape, z_dt=T.F32)
        T.tpmlp_device_status()
        assert bool((Z[M] == 7.0).all()) and bool((H[M] == 7.0).all()) and bool((ws[n:] == 0xFF).all())
        Zr, Hr = R.block_fwd(host(d["X"]), w, bb, host(d["bw"]) if bias else None, host(d["b2"]) if bias else None)
        U.assert_close(host(H[:M]), Hr, "bf16", "H")
        U.assert_close(host(Z[:M]), Zr, "bf16", "Z")
        assert torch.equal(Z32.to(torch.bfloat16), Z[:M])


@pytest.mark.parametrize("shape", BLOCKS + [(1, 31, 256, 256, 2), (32, 1, 256, 256, 2), (256, 1, 264, 256, 1), (512, 1, 256, 256, 1), (170, 5, 256, 128, 1)],
                         ids=lambda s: "s{}b{}h{}f{}p{}".format(*s))
def test_block_backward(T, shape, mode):
    import torch
    s, b, h, f, p = shape
    M = s * b
    d = make_block(T, *shape, seed=sum(shape) + 1)
    w, bb = R.q(host(d["W"])), R.q(host(d["B"]))
    H = bf16(np.random.default_rng(1).standard_normal((M, 2 * f)))
    new = lambda *shp, dt=torch.float32: torch.full(shp, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    dx, dw, db, dbw, db2 = R.block_bwd(host(d["X"]), w, bb, host(H), host(d["dZ"]))
    for grad_dt, tdt in ((T.F32, torch.float32), (T.BF16, torch.bfloat16)):
        dX, dW, dB = new(M, h, dt=torch.bfloat16), new(p, h, 2 * f // p, dt=tdt), new(f, h, dt=tdt)
        dbw_d, db2_d = new(p, 2 * f // p, dt=tdt), new(h, dt=tdt)
        ws, n = workspace(T, *shape, 1)
        T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, dbw_d, db2_d, ws, *shape, grad_dt=grad_dt)
        T.tpmlp_device_status()
        assert bool((ws[n:] == 0xFF).all())
        U.assert_close(host(dX), dx, "bf16", "dX")
        U.assert_close(host(dW.transpose(0, 1).reshape(h, 2 * f)), dw, "bf16", "dW")
        U.assert_close(host(dB), db, "bf16", "dB")
        U.assert_close(host(dbw_d).reshape(-1), dbw, "bf16", "dbw")
        U.assert_close(host(db2_d), db2, "bf16", "db2")
    # without the bias gradients, fp32 dX: the same bits otherwise
    dX32, dW2, dB2 = new(M, h), new(p, h, 2 * f // p, dt=torch.bfloat16), new(f, h, dt=torch.bfloat16)
    T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX32, dW2, dB2, None, None, ws, *shape, dx_dt=T.F32,
                                 grad_dt=T.BF16)
    T.tpmlp_device_status()
    assert torch.equal(dX32.to(torch.bfloat16), dX) and torch.equal(dW2, dW) and torch.equal(dB2, dB)


def test_block_backward_of_many_tiles(T):
    """Weight gradients and dX of more tiles than CTA pairs, dX's K loop the longest: the three products in one
    launch against one after the other (single CTAs), and against the reference."""
    import torch
    s, b, h, f, p = 201, 5, 1024, 4096, 4
    M = s * b
    d = make_block(T, s, b, h, f, p, seed=8)
    H = bf16(np.random.default_rng(2).standard_normal((M, 2 * f)))
    outs = []
    for md in (2, 0, 1):
        dX, dW, dB = torch.empty((M, h), device="cuda"), torch.empty((p, h, 2 * f // p), device="cuda"), torch.empty((f, h), device="cuda")
        ws, _ = workspace(T, s, b, h, f, p, 1)
        T.tpmlp_set_mxfp4_mode(md)
        try:
            T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, None, None, ws, s, b, h, f, p, dx_dt=T.F32)
            T.tpmlp_device_status()
        finally:
            T.tpmlp_set_mxfp4_mode(0)
        outs.append((dX, dW, dB))
    ref = R.block_bwd(host(d["X"]), R.q(host(d["W"])), R.q(host(d["B"])), host(H), host(d["dZ"]))
    for dX, dW, dB in outs:
        U.assert_close(host(dX), ref[0], "bf16", "dX")
        U.assert_close(host(dW.transpose(0, 1).reshape(h, 2 * f)), ref[1], "bf16", "dW")
        U.assert_close(host(dB), ref[2], "bf16", "dB")


def test_block_backward_same_bits_in_every_tiling(T):
    """Both tilings walk K in the same order without a split, so the backward's outputs are the same bits, run after
    run.  Large enough that every epilogue warp turns its buffers over many times (a copy that overtakes a read of
    the buffer it fills shows as a few wrong rows here)."""
    import torch
    s, b, h, f, p = 1024, 3, 512, 20480, 1
    M = s * b
    d = make_block(T, s, b, h, f, p, seed=4)
    H = torch.randn((M, 2 * f), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    want = None
    for md in (1, 2, 2, 2, 2, 0, 0):
        dX, dW, dB = torch.empty((M, h), device="cuda"), torch.empty((h, 2 * f), device="cuda"), torch.empty((f, h), device="cuda")
        dbw, db2 = torch.empty(2 * f, device="cuda"), torch.empty(h, device="cuda")
        ws, _ = workspace(T, s, b, h, f, p, 1)
        T.tpmlp_set_mxfp4_mode(md)
        try:
            T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, dbw, db2, ws, s, b, h, f, p, dx_dt=T.F32)
            T.tpmlp_device_status()
        finally:
            T.tpmlp_set_mxfp4_mode(0)
        got = (dX, dW, dB, dbw, db2)
        want = want or got
        for name, x, y in zip(("dX", "dW", "dB", "dbw", "db2"), want, got):
            assert torch.equal(x, y), (md, name, int((x != y).sum()))


def test_block_results_do_not_depend_on_p(T):
    """No scale block spans two shards, so the shard count changes the layout of dW and nothing else."""
    import torch
    s, b, h, f = 50, 3, 512, 1024
    outs = []
    for p in (1, 2, 4, 8):
        d = make_block(T, s, b, h, f, p, seed=77)
        Z = torch.empty((s * b, h), dtype=torch.bfloat16, device="cuda")
        H = torch.empty((s * b, 2 * f), dtype=torch.bfloat16, device="cuda")
        ws, _ = workspace(T, s, b, h, f, p, 0)
        T.tpmlp_mxfp4_swiglu_mlp_fwd(d["X"], *d["Wt"], d["bw"], *d["Bt"], d["b2"], Z, H, ws, s, b, h, f, p)
        dX, dW = torch.empty_like(Z), torch.empty((p, h, 2 * f // p), device="cuda")
        dB, dbw, db2 = torch.empty((f, h), device="cuda"), torch.empty(2 * f, device="cuda"), torch.empty(h, device="cuda")
        ws, _ = workspace(T, s, b, h, f, p, 1)
        T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, dbw, db2, ws, s, b, h, f, p)
        T.tpmlp_device_status()
        outs.append([Z, H, dX, dW.transpose(0, 1).reshape(h, 2 * f), dB, dbw, db2])
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], o))


def test_gradient_follows_differences_of_the_loss(T):
    """The backward's gradients against differences of the block's own loss <Z, dZ>: the forward on the GPU with
    X and the weights moved along the gradient.  The quantised forward is a staircase around the block, so
    the step is long (the values move by about their 4-bit step) and the two agree within the quantisation's noise:
    relative operand noise of about 0.1 a product over a few products, held to 0.3."""
    import torch
    s, b, h, f, p = 64, 4, 512, 1024, 2
    d = make_block(T, s, b, h, f, p, seed=5)
    M = s * b
    ws, _ = workspace(T, s, b, h, f, p, 0)
    H = torch.empty((M, 2 * f), dtype=torch.bfloat16, device="cuda")

    def loss(X, W, B):
        Wt, Bt = T.mxfp4_empty(2 * f, h), T.mxfp4_empty(h, f)
        W_sh = W.view(h, p, 2 * f // p).transpose(0, 1).contiguous()
        T.tpmlp_mxfp4_quantize(W_sh, None, None, *Wt, h, 2 * f, 2 * f // p, p, T.F32)
        T.tpmlp_mxfp4_quantize(B, None, None, *Bt, f, h, h, 1, T.F32)
        Z = torch.empty((M, h), device="cuda")
        T.tpmlp_mxfp4_swiglu_mlp_fwd(X.to(torch.bfloat16), *Wt, None, *Bt, None, Z, H, ws, s, b, h, f, p, z_dt=T.F32)
        return float((Z.double() * d["dZ"].double()).sum())

    X, W, B = d["X"].float(), d["W"].float(), d["B"].float().contiguous()
    loss(X, W, B)
    dX, dW, dB = torch.empty((M, h), device="cuda"), torch.empty((p, h, 2 * f // p), device="cuda"), torch.empty((f, h), device="cuda")
    wb, _ = workspace(T, s, b, h, f, p, 1)
    T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, None, None, wb, s, b, h, f, p, dx_dt=T.F32)
    T.tpmlp_device_status()
    dW = dW.transpose(0, 1).reshape(h, 2 * f)
    for name, v, g in (("X", X, dX), ("W", W, dW), ("B", B, dB)):
        step = 0.1 * v.norm() / g.norm()
        at = lambda t: loss(*(x + t * step * g if n == name else x for n, x in (("X", X), ("W", W), ("B", B))))  # noqa: E731
        diff = (at(1.0) - at(-1.0)) / 2
        want = float(step * g.double().square().sum())
        assert abs(diff - want) <= 0.3 * abs(want), (name, diff, want)


def test_block_on_another_stream_and_in_a_graph(T):
    import torch
    s, b, h, f, p = 9, 4, 256, 512, 2
    d = make_block(T, s, b, h, f, p, seed=21)
    ws, _ = workspace(T, s, b, h, f, p, 0)
    run = lambda Z: T.tpmlp_mxfp4_swiglu_mlp_fwd(d["X"], *d["Wt"], None, *d["Bt"], None, Z, None, ws, s, b, h, f, p)  # noqa: E731
    Z0, Z1, Z2 = (torch.zeros((s * b, h), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    run(Z0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(Z1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(Z2)
    Z2.zero_()
    graph.replay()
    T.tpmlp_device_status()
    assert torch.equal(Z0, Z1) and torch.equal(Z0, Z2)


def test_block_forward_right_after_its_weights_are_written(T):
    """The forward's kernels may start while the one ahead ends; weights written just before a call are the ones it uses."""
    import torch
    s, b, h, f, p = 4, 1, 512, 1024, 1
    two = [make_block(T, s, b, h, f, p, seed=31 + i) for i in range(2)]
    ws, _ = workspace(T, s, b, h, f, p, 0)
    X = two[0]["X"]
    want = []
    for d in two:
        Z = torch.empty((s, h), dtype=torch.bfloat16, device="cuda")
        T.tpmlp_mxfp4_swiglu_mlp_fwd(X, *d["Wt"], None, *d["Bt"], None, Z, None, ws, s, b, h, f, p)
        torch.cuda.synchronize()
        want.append(Z)
    assert not torch.equal(*want)
    W, Wt, Bt = torch.empty_like(two[0]["W"]), T.mxfp4_empty(2 * f, h), T.mxfp4_empty(h, f)
    Z = torch.empty((40, s, h), dtype=torch.bfloat16, device="cuda")
    for i in range(40):
        d = two[i % 2]
        if i % 4 < 2:  # by copies, or by the quantiser with a copy ahead of it
            for dst, src in zip(Wt + Bt, d["Wt"] + d["Bt"]):
                dst.copy_(src)
        else:
            W.copy_(d["W"])
            T.tpmlp_mxfp4_quantize(d["B"], None, None, *Bt, f, h, h)
            T.tpmlp_mxfp4_quantize(W, None, None, *Wt, h, 2 * f, 2 * f)
        T.tpmlp_mxfp4_swiglu_mlp_fwd(X, *Wt, None, *Bt, None, Z[i], None, ws, s, b, h, f, p)
    T.tpmlp_device_status()
    for i in range(40):
        assert torch.equal(Z[i], want[i % 2]), i


def test_bases_aligned_to_16_bytes_only(T, mode):
    """Every tensor 16 bytes into an allocation: 32-byte accesses must give way."""
    import torch
    s, b, h, f, p = 37, 4, 256, 512, 2
    M = s * b

    def at16(t):
        n = t.numel() * t.element_size()
        raw = torch.zeros(n + 16, dtype=torch.uint8, device="cuda")
        v = raw[16:].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    d = make_block(T, s, b, h, f, p, seed=12)
    e = {k: tuple(at16(x) for x in v) if isinstance(v, tuple) else at16(v) for k, v in d.items()}
    outs = []
    for x, put in ((d, lambda t: t), (e, at16)):
        Z, H = put(torch.zeros_like(x["X"])), put(torch.zeros((M, 2 * f), dtype=torch.bfloat16, device="cuda"))
        ws = put(workspace(T, s, b, h, f, p, 0)[0])
        T.tpmlp_mxfp4_swiglu_mlp_fwd(x["X"], *x["Wt"], x["bw"], *x["Bt"], x["b2"], Z, H, ws, s, b, h, f, p)
        dX, dW, dB = put(torch.zeros_like(x["X"])), put(torch.zeros((p, h, 2 * f // p), device="cuda")), put(torch.zeros((f, h), device="cuda"))
        dbw, db2 = put(torch.zeros(2 * f, device="cuda")), put(torch.zeros(h, device="cuda"))
        ws = put(workspace(T, s, b, h, f, p, 1)[0])
        T.tpmlp_mxfp4_swiglu_mlp_bwd(x["X"], *x["Wn"], *x["Bn"], H, x["dZ"], dX, dW, dB, dbw, db2, ws, s, b, h, f, p)
        T.tpmlp_device_status()
        outs.append((Z, H, dX, dW, dB, dbw, db2))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_offsets_past_32_bits(T):
    """Tensors of more than 2^31 values: what lies at their far end is right."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = 24  # rows looked at
    rows, cols = 270_001, 8192
    X = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=gen)
    a, t = T.mxfp4_empty(rows, cols), T.mxfp4_empty(cols, rows)
    T.tpmlp_mxfp4_quantize(X, *a, *t, rows, cols, cols)
    codes, sc = R.quantize(host(X[-n:]))
    assert np.array_equal(a[0][-n:].cpu().numpy(), codes)
    got = R.untile_scales(a[1][-1:].cpu().numpy(), rows - (rows - 1) // 128 * 128, cols)
    assert np.array_equal(got[-min(n, got.shape[0]):], sc[-min(n, got.shape[0]):])
    codes, _ = R.quantize(host(X[:, -n:]).T)
    assert np.array_equal(t[0][-n:].cpu().numpy(), codes)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    T.tpmlp_mxfp4_dequantize(*a, out, rows, cols)
    assert np.array_equal(host(out[-n:]), R.q(host(X[-n:])))
    del X, a, t, out
    # product: D of 2.2e9 values
    m, k = 540_000, 64
    A = torch.randn((m, k), generator=gen, device="cuda").to(torch.bfloat16)
    B = torch.randn((4096, k), generator=gen, device="cuda").to(torch.bfloat16)
    aq, bq = T.mxfp4_empty(m, k), T.mxfp4_empty(4096, k)
    T.tpmlp_mxfp4_quantize(A, *aq, None, None, m, k, k)
    T.tpmlp_mxfp4_quantize(B, *bq, None, None, 4096, k, k)
    D = torch.empty((m, 4096), dtype=torch.bfloat16, device="cuda")
    T.tpmlp_mxfp4_matmul(*aq, *bq, None, D, m, 4096, k)
    R.assert_product(host(D[-n:]), R.q(host(A[-n:])), R.q(host(B)))
    del A, D
    # block: pre-activations of 2.3e9 values
    s, b, h, f, p = 55_001, 1, 256, 20480, 2
    d = make_block(T, s, b, h, f, p, seed=30)
    Z, H = torch.empty((s, h), dtype=torch.bfloat16, device="cuda"), torch.empty((s, 2 * f), dtype=torch.bfloat16, device="cuda")
    ws, _ = workspace(T, s, b, h, f, p, 0)
    T.tpmlp_mxfp4_swiglu_mlp_fwd(d["X"], *d["Wt"], d["bw"], *d["Bt"], d["b2"], Z, H, ws, s, b, h, f, p)
    Zr, Hr = R.block_fwd(host(d["X"][-n:]), R.q(host(d["W"]).T), R.q(host(d["B"]).T), host(d["bw"]), host(d["b2"]))
    U.assert_close(host(H[-n:]), Hr, "bf16", "H")
    U.assert_close(host(Z[-n:]), Zr, "bf16", "Z")
    dX, dW, dB = torch.empty_like(Z), torch.empty((p, h, 2 * f // p), device="cuda"), torch.empty((f, h), device="cuda")
    dbw, db2 = torch.empty(2 * f, device="cuda"), torch.empty(h, device="cuda")
    ws, _ = workspace(T, s, b, h, f, p, 1)
    T.tpmlp_mxfp4_swiglu_mlp_bwd(d["X"], *d["Wn"], *d["Bn"], H, d["dZ"], dX, dW, dB, dbw, db2, ws, s, b, h, f, p)
    T.tpmlp_device_status()
    dXr = R.block_bwd(host(d["X"][-n:]), R.q(host(d["W"])), R.q(host(d["B"])), host(H[-n:]), host(d["dZ"][-n:]))[0]
    U.assert_close(host(dX[-n:]), dXr, "bf16", "dX")
    U.assert_close(host(db2), d["dZ"].double().sum(0).cpu().numpy(), "bf16", "db2")


def test_empty_batch_writes_nothing(T):
    import torch
    n0 = T.tpmlp_launch_count()
    t = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    o = torch.full((512,), 5.0, device="cuda")
    T.tpmlp_mxfp4_matmul(t, t[512:], t[1024:], t[2048:], None, o, 0, 8, 32, T.F32)
    T.tpmlp_mxfp4_quantize(t, t[512:], t[1024:], None, None, 0, 32, 32)
    T.tpmlp_mxfp4_dequantize(t, t[512:], o, 0, 32, T.F32)
    torch.cuda.synchronize()
    assert T.tpmlp_launch_count() == n0 and bool((o == 5.0).all())


def test_example_trains_and_serves(T):
    """The example's block learns, and single tokens give the batch's rows: to the bf16 store (a row is quantised by
    itself, the kernels for one token and for many differ in fp32 summation order only) up to a rounding of Y that
    falls the other way, 2e-2 of the outputs' size."""
    from megatron_tensor_mlp_gb300 import mxfp4_block
    losses, served, batch = mxfp4_block.train_and_serve()
    assert losses[-1] < 0.5 * losses[0], losses
    a, b = host(served), host(batch)
    assert np.max(np.abs(a - b)) <= 2e-2 * np.sqrt(np.mean(b * b)) + R.half_spacing(np.max(np.abs(b)), 8) * 2
