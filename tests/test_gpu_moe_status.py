"""A plan that had to be cut is reported, and changes nothing for the other calls of its device."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import moe_ref as R  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


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


def cut_plan(T):
    """A row range past the rows: cut in the kernel, recorded, not yet read."""
    x, w, y = rnd(8, 64), rnd(2, 64, 128), torch.zeros(8, 128, dtype=BF, device="cuda")
    T.tpmlp_moe_matmul(x, None, torch.tensor([0, 6, 9], dtype=I32, device="cuda"), w, None, y, None, 8, 8, 2, 64, 128)


def test_a_timeout_behind_a_cut_plan_is_not_lost(T):
    cut_plan(T)
    T.tpmlp_debug_wait_timeout(20000)
    assert T.tpmlp_device_status(check=False) == T.ERR_TIMEOUT
    assert "plan" in T.last_error()  # both are named
    assert T.tpmlp_device_status(check=False) == T.OK
    T.tpmlp_debug_wait_timeout(20000)
    cut_plan(T)
    assert T.tpmlp_device_status(check=False) == T.ERR_TIMEOUT
    assert T.tpmlp_device_status(check=False) == T.OK
    cut_plan(T)
    assert T.tpmlp_device_status(check=False) == T.ERR_DEVICE
    assert T.tpmlp_device_status(check=False) == T.OK


@pytest.mark.parametrize("kind", ["column", "experts", "mxfp4"])
def test_a_cut_plan_ends_no_other_call(T, kind):
    """Products of one tile and a long contraction, in which every role waits for many milliseconds, give the same bits while a cut
    plan is recorded and not yet read."""
    m, n = 256, 256
    k = 1 << (18 if kind == "mxfp4" else 21)
    x, w = rnd(m, k), rnd(n, k, seed=1) if kind == "mxfp4" else rnd(k, n, seed=1)
    if kind == "mxfp4":
        a, b = T.mxfp4_empty(m, k), T.mxfp4_empty(n, k)
        T.tpmlp_mxfp4_quantize(x, *a, None, None, m, k, k)
        T.tpmlp_mxfp4_quantize(w, *b, None, None, n, k, k)
    off = torch.tensor([0, m], dtype=I32, device="cuda")

    def product():
        y = torch.full((m, n), float("nan"), dtype=BF, device="cuda")
        if kind == "column":
            T.tpmlp_column_fwd(x, w, None, y, None, m, 1, k, n, 1, act=T.ACT_NONE)
        elif kind == "experts":
            T.tpmlp_moe_matmul(x, None, off, w, None, y, None, m, m, 1, k, n)
        else:
            T.tpmlp_mxfp4_matmul(*a, *b, None, y, m, n, k)
        return y

    want = product()
    assert T.tpmlp_device_status(check=False) == T.OK
    assert torch.isfinite(want).all()
    cut_plan(T)
    got = product()
    assert T.tpmlp_device_status(check=False) == T.ERR_DEVICE
    assert torch.equal(got, want)


@pytest.mark.parametrize("what", ["range", "falling", "token", "weight gradient"])
def test_every_kind_of_cut_is_reported_once(T, what):
    """By the kernel for few rows and by those of CTA pairs."""
    for rows, e in ((40, 8), (900, 2)):
        K, N = 64, 520
        x, w, y = rnd(rows, K), rnd(e, K, N), torch.zeros(rows, N, dtype=BF, device="cuda")
        at = [rows * i // e for i in range(e + 1)]
        src = torch.arange(rows, dtype=I32, device="cuda")
        if what == "range":
            at[-1] += 3
        elif what == "falling":
            at[1] = at[2] + 1
        else:
            src[rows // 2] = rows
        off = torch.tensor(at, dtype=I32, device="cuda")
        if what == "weight gradient":
            dw = torch.empty(e, K, N, dtype=BF, device="cuda")
            T.tpmlp_moe_matmul_dw(x, src, off, y, dw, None, rows, rows, e, K, N, grad_dt=0)
        else:
            T.tpmlp_moe_matmul(x, src if what == "token" else None, off, w, None, y, None, rows, rows, e, K, N)
        assert T.tpmlp_device_status(check=False) == T.ERR_DEVICE
        assert T.tpmlp_device_status(check=False) == T.OK
