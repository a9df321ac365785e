"""Layer norm of columns of one tensor into other columns of it, on the GPU: the bits of tensors of their own."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,h", [(1, 64), (37, 1001), (37, 1024), (1300, 3080), (700, 8192)])
def test_columns_of_one_tensor(rows, h, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import tpmlp as T
    g = torch.Generator(device="cuda").manual_seed(h)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    dt, ld = 0 if dtype == BF else 1, 4 * h
    x, dy, gamma, beta = n(rows, h), n(rows, h), n(h), n(h)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    stats = [torch.empty(rows, device="cuda") for _ in range(4)]
    sums = [torch.empty(h, device="cuda") for _ in range(4)]
    ws = torch.empty(T.tpmlp_layernorm_ws_bytes(rows, h), dtype=torch.uint8, device="cuda")
    T.tpmlp_layernorm_fwd(x, gamma, beta, y, *stats[:2], rows, h, h, h, 1e-5, dt)
    T.tpmlp_layernorm_bwd(x, gamma, *stats[:2], dy, dx, *sums[:2], ws, rows, h, h, h, h, dt, 1)
    room = torch.full((rows, ld), 7.0, dtype=dtype, device="cuda")  # dx | x | dy | y
    parts = room[:, :h], room[:, h:2 * h], room[:, 2 * h:3 * h], room[:, 3 * h:]
    parts[1].copy_(x)
    parts[2].copy_(dy)
    T.tpmlp_layernorm_fwd(parts[1], gamma, beta, parts[3], *stats[2:], rows, h, ld, ld, 1e-5, dt)
    T.tpmlp_layernorm_bwd(parts[1], gamma, *stats[2:], parts[2], parts[0], *sums[2:], ws, rows, h, ld, ld, ld, dt, 1)
    for got, want in zip(parts, (dx, x, dy, y)):
        assert torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(stats[2:] + sums[2:], stats[:2] + sums[:2]))
