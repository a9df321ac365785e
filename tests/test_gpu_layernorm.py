"""Layer norm forward and backward on the GPU, against 64 bits (tests/moe_ref.py)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import moe_ref as R  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import tpmlp
    yield tpmlp
    tpmlp.tpmlp_device_status()


def data(rows, h, dtype, seed=0, mean=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (n(rows, h) * torch.exp(n(1, h) * 0.5) + mean).to(dtype)
    return x, (1 + 0.3 * n(h)).to(dtype), (0.2 * n(h)).to(dtype), n(rows, h).to(dtype)


# A sum of h terms: at most 32 in a thread and 16 across threads, each a rounding of 2^-24 of the magnitudes.
SUM = 48 * 2.0**-24


def fwd_slack(x, gamma, rstd, mean):
    """mean is off by SUM of the mean magnitude, the difference and rstd by a few roundings more."""
    x = x.to(R.D)
    size = (x.abs() + x.abs().mean(1, keepdim=True) * 2) * rstd[:, None]
    n = (x - mean[:, None]).abs() * rstd[:, None]
    g = 1.0 if gamma is None else gamma.to(R.D).abs()
    return (SUM * size + SUM * n) * g


WIDTHS = [1, 8, 31, 64, 256, 1000, 1001, 1024, 1032, 2056, 4097, 5120, 8192, 8200, 16384, 16383]


@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_and_backward(T, h, dtype):
    rows, dt = 37, 0 if dtype == BF else 1
    x, gamma, beta, dy = data(rows, h, dtype, seed=h)
    y = torch.full_like(x, NAN)
    mean, rstd = torch.full((rows,), NAN, device="cuda"), torch.full((rows,), NAN, device="cuda")
    T.tpmlp_layernorm_fwd(x, gamma, beta, y, mean, rstd, rows, h, h, h, 1e-5, dt)
    ry, rm, rr = R.norm(x, gamma, beta, 1e-5)
    R.close(mean, rm, SUM * x.to(R.D).abs().mean(1), "mean")
    # variance: relative error SUM, and the mean's own error squared (rows of one value: rstd is 1 / sqrt(eps))
    e2 = (SUM * x.to(R.D).abs().amax(1)) ** 2
    R.close(rstd, rr, rr * (SUM + e2 * rr * rr), "rstd")
    R.close(y, ry, fwd_slack(x, gamma, rr, rm) + 2.0**-23 * beta.to(R.D).abs(), "y")
    dx, dg, db = torch.full_like(x, NAN), torch.full((h,), NAN, device="cuda"), torch.full((h,), NAN, device="cuda")
    ws = torch.empty(T.tpmlp_layernorm_ws_bytes(rows, h), dtype=torch.uint8, device="cuda")
    T.tpmlp_layernorm_bwd(x, gamma, mean, rstd, dy, dx, dg, db, ws, rows, h, h, h, h, dt, 1)
    rdx, rdg, rdb = R.norm_bwd(x, gamma, mean, rstd, dy)
    m, s = mean.to(R.D)[:, None], rstd.to(R.D)[:, None]
    xhat, g = (x.to(R.D) - m).abs() * s, (dy.to(R.D) * gamma.to(R.D)).abs()
    size = s * (g + g.mean(1, keepdim=True) + xhat * (g * xhat).mean(1, keepdim=True))
    R.close(dx, rdx, 2 * SUM * size, "dx")
    R.close(dg, rdg, SUM * (dy.to(R.D).abs() * xhat).sum(0), "dgamma")
    R.close(db, rdb, SUM * dy.to(R.D).abs().sum(0), "dbeta")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,h", [(1, 5120), (3, 64), (1000, 72), (5000, 136), (1303, 1001), (2500, 1024), (1300, 1032), (1001, 3080),
                                    (1001, 5120), (700, 8192), (700, 12288), (650, 16384), (650, 5121)])
def test_row_counts_and_gradient_types(T, rows, h, dtype):
    """More rows than CTAs, fewer rows than CTAs; bf16 gradients; one of the two sums."""
    dt = 0 if dtype == BF else 1
    x, gamma, _, dy = data(rows, h, dtype, seed=rows)
    _, rm, rr = R.norm(x, None, None, 1e-5)
    mean, rstd = rm.float(), rr.float()
    rdx, rdg, rdb = R.norm_bwd(x, gamma, mean, rstd, dy)
    ws = torch.empty(T.tpmlp_layernorm_ws_bytes(rows, h), dtype=torch.uint8, device="cuda")
    # rows / 152 in a thread, 8 warps, up to 608 / 16 parts, 16 at the end
    slack = (rows / 152 + 64) * 2.0**-24
    xhat = (x.to(R.D) - mean.to(R.D)[:, None]).abs() * rstd.to(R.D)[:, None]
    sizes = (dy.to(R.D).abs() * xhat).sum(0), dy.to(R.D).abs().sum(0)
    for grad in (BF, F32):
        dx, dg, db = torch.empty_like(x), *(torch.full((h,), NAN, dtype=grad, device="cuda") for _ in range(2))
        T.tpmlp_layernorm_bwd(x, gamma, mean, rstd, dy, dx, dg, None, ws, rows, h, h, h, h, dt, 0 if grad == BF else 1)
        R.close(dg, rdg, slack * sizes[0], "dgamma")
        T.tpmlp_layernorm_bwd(x, gamma, mean, rstd, dy, dx, None, db, ws, rows, h, h, h, h, dt, 0 if grad == BF else 1)
        R.close(db, rdb, slack * sizes[1], "dbeta")
    dx2 = torch.full_like(x, NAN)
    T.tpmlp_layernorm_bwd(x, gamma, mean, rstd, dy, dx2, None, None, None, rows, h, h, h, h, dt, 1)
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ld,shift", [(1040, 0), (1043, 0), (1040, 1), (1024, 8)])
def test_strides_and_alignment(T, ld, shift, dtype):
    """Rows with a pitch, at a base that is aligned to an element only; what lies between the rows stays."""
    rows, h, dt = 19, 1024, 0 if dtype == BF else 1
    x, gamma, beta, dy = data(rows, h, dtype, seed=1)
    pad = lambda t: torch.full((rows * ld + shift,), 7.0, dtype=dtype, device="cuda")[shift:].view(rows, ld) if t is None else _put(pad(None), t)  # noqa: E731

    def _put(room, t):
        room[:, :h] = t
        return room

    xs, dys, ys, dxs = pad(x), pad(dy), pad(None), pad(None)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    T.tpmlp_layernorm_fwd(x, gamma, beta, y, mean, rstd, rows, h, h, h, 1e-5, dt)
    T.tpmlp_layernorm_fwd(xs, gamma, beta, ys, None, None, rows, h, ld, ld, 1e-5, dt)
    ry, rm, rr = R.norm(x, gamma, beta, 1e-5)
    slack = fwd_slack(x, gamma, rr, rm) + 2.0**-23 * beta.to(R.D).abs()
    R.close(ys[:, :h], ry, slack, "y")
    R.close(y, ry, slack, "y")
    T.tpmlp_layernorm_bwd(xs, gamma, mean, rstd, dys, dxs, None, None, None, rows, h, ld, ld, ld, dt, 1)
    rdx, _, _ = R.norm_bwd(x, gamma, mean, rstd, dy)
    s = rstd.to(R.D)[:, None]
    xhat, g = (x.to(R.D) - mean.to(R.D)[:, None]).abs() * s, (dy.to(R.D) * gamma.to(R.D)).abs()
    R.close(dxs[:, :h], rdx, 2 * SUM * s * (g + g.mean(1, keepdim=True) + xhat * (g * xhat).mean(1, keepdim=True)), "dx")
    if ld > h:
        assert (ys[:, h:] == 7.0).all() and (dxs[:, h:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,h", [(1900, 1032), (1000, 3080), (1300, 3608), (1301, 4096), (1300, 4104), (1001, 5120), (700, 8192),
                                    (700, 12288), (400, 14336), (401, 16384)])
def test_many_wide_rows(T, rows, h, dtype):
    """More rows than CTAs, which go through a ring in shared memory: with a pitch, without gamma or beta too."""
    dt, ld = 0 if dtype == BF else 1, h + 8
    x, gamma, beta, dy = data(rows, h, dtype, seed=h)
    room = lambda t=None: torch.full((rows, ld), 7.0, dtype=dtype, device="cuda") if t is None else torch.nn.functional.pad(t, (0, 8), value=7.0)  # noqa: E731
    xs, dys = room(x), room(dy)
    for g, b in ((gamma, beta), (None, None), (gamma, None)):
        y, dx = room(), room()
        mean, rstd = torch.full((rows,), NAN, device="cuda"), torch.full((rows,), NAN, device="cuda")
        T.tpmlp_layernorm_fwd(xs, g, b, y, mean, rstd, rows, h, ld, ld, 1e-5, dt)
        ry, rm, rr = R.norm(x, g, b, 1e-5)
        R.close(mean, rm, SUM * x.to(R.D).abs().mean(1), "mean")
        R.close(rstd, rr, rr * (SUM + (SUM * x.to(R.D).abs().amax(1) * rr) ** 2), "rstd")
        R.close(y[:, :h], ry, fwd_slack(x, g, rr, rm) + 2.0**-23 * (0 if b is None else b.to(R.D).abs()), "y")
        T.tpmlp_layernorm_bwd(xs, g, mean, rstd, dys, dx, None, None, None, rows, h, ld, ld, ld, dt, 1)
        rdx, _, _ = R.norm_bwd(x, g, mean, rstd, dy)
        s = rstd.to(R.D)[:, None]
        xhat, gg = (x.to(R.D) - mean.to(R.D)[:, None]).abs() * s, (dy.to(R.D) * (1 if g is None else g.to(R.D))).abs()
        R.close(dx[:, :h], rdx, 2 * SUM * s * (gg + gg.mean(1, keepdim=True) + xhat * (gg * xhat).mean(1, keepdim=True)), "dx")
        assert (y[:, h:] == 7.0).all() and (dx[:, h:] == 7.0).all()


def test_without_gamma_and_beta(T):
    rows, h = 11, 520
    x, gamma, beta, dy = data(rows, h, BF)
    y, y1 = torch.empty_like(x), torch.empty_like(x)
    one, zero = torch.ones(h, dtype=BF, device="cuda"), torch.zeros(h, dtype=BF, device="cuda")
    T.tpmlp_layernorm_fwd(x, None, None, y, None, None, rows, h, h, h)
    T.tpmlp_layernorm_fwd(x, one, zero, y1, None, None, rows, h, h, h)
    assert torch.equal(y, y1)
    _, m, r = R.norm(x, None, None, 1e-5)
    T.tpmlp_layernorm_bwd(x, None, m.float(), r.float(), dy, y, None, None, None, rows, h, h, h, h)
    T.tpmlp_layernorm_bwd(x, one, m.float(), r.float(), dy, y1, None, None, None, rows, h, h, h, h)
    assert torch.equal(y, y1)


def test_rows_of_one_value_and_not_finite(T):
    """A constant row has no spread: y is beta.  A NaN or an infinity stays in its row."""
    rows, h = 6, 1024
    x, gamma, beta, _ = data(rows, h, F32)
    x[0], x[1, 5], x[2, 7] = 3.0, NAN, float("inf")
    y = torch.empty_like(x)
    T.tpmlp_layernorm_fwd(x, gamma, beta, y, None, None, rows, h, h, h, 1e-5, 1)
    assert torch.equal(y[0], beta)
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[2]).any() and torch.isfinite(y[3:]).all()


def test_no_rows(T):
    dg, db = torch.full((64,), NAN, device="cuda"), torch.full((64,), NAN, device="cuda")
    T.tpmlp_layernorm_fwd(None, None, None, None, None, None, 0, 64, 64, 64)
    T.tpmlp_layernorm_bwd(None, None, None, None, None, None, dg, db, None, 0, 64, 64, 64, 64)
    assert (dg == 0).all() and (db == 0).all()


def test_same_bits_every_time(T):
    rows, h = 3000, 1000
    x, gamma, beta, dy = data(rows, h, BF)
    mean, rstd = x.float().mean(1), torch.rsqrt(x.float().var(1, unbiased=False) + 1e-5)
    ws = torch.empty(T.tpmlp_layernorm_ws_bytes(rows, h), dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0, 255):
        ws.fill_(fill)
        o = torch.empty_like(x), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
        T.tpmlp_layernorm_bwd(x, gamma, mean, rstd, dy, *o, ws, rows, h, h, h, h)
        outs.append(o)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
