"""Layer norm of rows whose mean is large against their spread, on the GPU, against 64 bits (tests/moe_ref.py)."""
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


def forward(T, x, gamma, beta):
    rows, h = x.shape
    y = torch.full_like(x, NAN)
    mean, rstd = torch.full((rows,), NAN, device="cuda"), torch.full((rows,), NAN, device="cuda")
    T.tpmlp_layernorm_fwd(x, gamma, beta, y, mean, rstd, rows, h, h, h, 1e-5, 0 if x.dtype == BF else 1)
    return y, mean, rstd


# Widths whose reciprocal is rounded, on a warp, on a CTA, element by element and, with many rows, through the ring.
SIZES = [(5, 1000), (700, 1000), (5, 1001), (700, 1001), (5, 3840), (1300, 3840), (5, 4095), (5, 15360), (400, 15360)]
# A sum of h terms: at most 32 in a thread and 16 across threads, each a rounding of 2^-24 of the magnitudes.
SUM = 48 * 2.0**-24


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,h", SIZES)
def test_a_constant_row_is_beta(T, rows, h, dtype):
    """No spread, whatever the value: y is beta to the bit, the mean the value, rstd 1 / sqrt(eps)."""
    g = torch.Generator(device="cuda").manual_seed(h)
    gamma, beta = (torch.randn(h, generator=g, device="cuda").to(dtype) for _ in range(2))
    values = torch.tensor([3.0, -3.0, 1000.0, 3008.0, 0.0, 2.0**-10, -77.0], device="cuda")
    x = values[torch.arange(rows, device="cuda") % 7][:, None].expand(rows, h).to(dtype).contiguous()
    y, mean, rstd = forward(T, x, gamma, beta)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, beta.expand(rows, h))
    # rsqrt is within 2 units in the last place, eps and the sum are roundings of their own
    assert ((rstd.to(R.D) * 1e-5**0.5 - 1).abs() <= 4 * 2.0**-23).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,h", SIZES)
@pytest.mark.parametrize("value", [3.0, 1000.0, 3008.0, -60000.0])
def test_a_small_spread_on_a_large_mean(T, rows, h, dtype, value):
    """The error goes by the differences from the mean, not by the values."""
    g = torch.Generator(device="cuda").manual_seed(h)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gamma, beta = (1 + 0.3 * n(h)).to(dtype), (0.2 * n(h)).to(dtype)
    # bf16 cannot hold a spread below its own step: a few values one step away
    if dtype == BF:
        step = 2.0 ** (torch.tensor(abs(value)).log2().floor().item() - 7)
        x = (value + step * (torch.rand(rows, h, generator=g, device="cuda") < 0.01)).to(dtype)
    else:
        x = value + abs(value) * 1e-6 * n(rows, h)
    y, mean, rstd = forward(T, x, gamma, beta)
    ry, rm, rr = R.norm(x, gamma, beta, 1e-5)
    delta = (x.to(R.D) - rm[:, None]).abs()
    size = delta.mean(1, keepdim=True)
    # The first mean m0 is off by E.  A difference d = x - m0 is rounded once (2^-24 |d|, |d| <= delta + E); its mean, by which
    # m0 is corrected, is off by SUM of the mean |d|; the corrected difference is rounded once more.
    E = SUM * x.to(R.D).abs().mean(1, keepdim=True) * 1.1
    off = SUM * (size + E)
    diff = 2.0**-24 * (2 * delta + 2 * E) + off
    R.close(mean, rm, off[:, 0], "mean")
    # the variance: a sum of d^2, at most delta^2 + E^2 in the mean, and its correction
    rel = SUM * ((delta**2).mean(1) + 2 * E[:, 0] ** 2) * rr**2 + 4 * 2.0**-24
    R.close(rstd, rr, rr * rel, "rstd")
    s, unit = rr[:, None], delta * rr[:, None]
    R.close(y, ry, ((diff * s + unit * rel[:, None]) * (1 + rel[:, None]) + 2.0**-23 * unit) * gamma.to(R.D).abs()
            + 2.0**-23 * beta.to(R.D).abs(), "y")


def test_an_infinity_keeps_the_mean_and_overflowing_squares_the_finite_outputs(T):
    """What large values gave before: a row with an infinity has that mean, squares past the range have rstd 0 and y beta."""
    rows, h = 3, 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows, h, generator=g, device="cuda")
    beta = torch.randn(h, generator=g, device="cuda")
    x[0, 7], x[1] = float("inf"), x[1] * 2.0**80
    y, mean, rstd = forward(T, x, None, beta)
    assert mean[0] == float("inf") and torch.isnan(rstd[0]) and torch.isnan(y[0]).all()
    assert rstd[1] == 0 and torch.equal(y[1], beta)
    assert torch.isfinite(y[2]).all()
