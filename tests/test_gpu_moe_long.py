"""Weight gradients of experts with very many rows, on the GPU, against 64 bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import moe_ref as R  # noqa: E402

BF, F32, I32, D = torch.bfloat16, torch.float32, torch.int32, torch.float64
CHUNK = 262144  # rows that are added in one accumulator


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import tpmlp
    yield tpmlp
    tpmlp.tpmlp_device_status()


def positive(*shape, seed=0):
    return (torch.rand(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") + 0.5).to(BF)


@pytest.mark.parametrize("counts,K,N,gathered", [([2097152 - 77, 0, 5, 3 * CHUNK], 72, 136, False), ([CHUNK, CHUNK + 1, 40, 2 * CHUNK - 64], 136, 72, True),
                                                 ([700001], 8, 264, False), ([100, 600001], 264, 1544, True)])
def test_sums_over_millions_of_rows(T, counts, K, N, gathered):
    """Terms of one sign, whose sums' errors add up too: at most 2^-23 of the running sum for each 16 terms (moe_ref.py), which is
    at most the chunk's, so (CHUNK / 16 + 16) 2^-23 = 2.0e-3 of it; the chunks' sums are added with a rounding each.  (In one
    accumulation 700001 rows are 4.6e-3 off.)"""
    e, rows = len(counts), sum(counts) + 3
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=I32, device="cuda")
    tokens = rows // 3 if gathered else rows
    x, dy = positive(tokens, K, seed=1), positive(rows, N, seed=2)
    src = torch.randint(0, tokens, (rows,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda", dtype=I32) if gathered else None
    dw, db = torch.full((e, K, N), float("nan"), device="cuda"), torch.full((e, N), float("nan"), device="cuda")
    T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, tokens, rows, e, K, N)
    for i in range(e):
        a, b = int(off[i]), int(off[i + 1])
        ref, sums = torch.zeros(K, N, dtype=D, device="cuda"), torch.zeros(N, dtype=D, device="cuda")
        for c in range(a, b, CHUNK):
            at = slice(c, min(c + CHUNK, b))
            xs = x[at] if src is None else x[src[at].long()]
            ref += xs.to(D).t() @ dy[at].to(D)
            sums += dy[at].to(D).sum(0)
        n = -(-(b - a) // CHUNK)
        bound = R.product_bound(min(b - a, CHUNK)) + n * 2.0**-24
        assert ((dw[i].to(D) - ref).abs() <= ref * bound * (1 + 2.0**-8)).all(), i
        # a lane adds every 128th row, then 4 lanes and 32 warps
        assert ((db[i].to(D) - sums).abs() <= sums * ((b - a) / 128 + 64) * 2.0**-24).all(), i
    again = torch.full_like(dw, float("nan"))
    T.tpmlp_moe_matmul_dw(x, src, off, dy, again, None, tokens, rows, e, K, N)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("k_blocks", [1, 2, 7])
@pytest.mark.parametrize("K,N,gathered", [(72, 136, False), (264, 520, True), (200, 1544, True)])
def test_short_chunks(T, k_blocks, K, N, gathered):
    """Chunks of 64 rows and more: whole numbers, whose sums are exact in any order; experts without rows, of a chunk's rows,
    one more and one less.  bf16 gradients are not split."""
    counts = [0, 1, 64, 65, 63, 128, 0, 449, 300, 7]
    e, n = len(counts), sum(counts)
    rows = n + 5
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=I32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(k_blocks)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(BF)  # noqa: E731
    tokens = rows // 2 if gathered else rows
    src = torch.randint(0, tokens, (rows,), generator=g, device="cuda", dtype=I32) if gathered else None
    x, dy = whole(tokens, K), whole(rows, N)
    dy[n:] = float("nan")
    if not gathered:
        x[n:] = float("nan")
    xs = (x if src is None else x[src.long()])[:n]
    ref, _, sums, _ = R.dw(xs, off, dy[:n], e)
    T.tpmlp_set_k_chunk(k_blocks)
    try:
        dw, db = torch.full((e, K, N), float("nan"), device="cuda"), torch.full((e, N), float("nan"), device="cuda")
        T.tpmlp_moe_matmul_dw(x, src, off, dy, dw, db, tokens, rows, e, K, N)
        assert torch.equal(dw.to(D), ref) and torch.equal(db.to(D), sums)
        half = torch.full((e, K, N), float("nan"), dtype=BF, device="cuda")
        T.tpmlp_moe_matmul_dw(x, src, off, dy, half, None, tokens, rows, e, K, N, grad_dt=0)
        assert torch.equal(half, ref.to(F32).to(BF))
    finally:
        T.tpmlp_set_k_chunk(0)
