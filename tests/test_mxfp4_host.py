"""MXFP4 operators on the host: sizes, refusals before any CUDA call, and the gradient's formula against
differences in 64 bits (CPU only)."""
import numpy as np
import pytest

import mxfp4_ref as R
from megatron_tensor_mlp_gb300 import build as B

B.build()
from megatron_tensor_mlp_gb300 import tpmlp as T  # noqa: E402

MB = 0x1000000


def addr(i):
    """16-byte aligned addresses 16 MB apart that are never dereferenced."""
    return 0x7F0000000000 + i * MB


def test_sizes():
    assert T.tpmlp_mxfp4_code_bytes(3, 1) == 48 and T.tpmlp_mxfp4_code_bytes(3, 33) == 96
    assert T.tpmlp_mxfp4_scale_bytes(1, 1) == 512 and T.tpmlp_mxfp4_scale_bytes(129, 129) == 2048
    assert T.tpmlp_mxfp4_code_bytes(-1, 32) == -1 and T.tpmlp_mxfp4_scale_bytes(4, 0) == -1
    assert T.tpmlp_mxfp4_swiglu_ws_bytes(4, 2, 64, 256, 2) > 0
    assert T.tpmlp_mxfp4_swiglu_ws_bytes(4, 2, 64, 192, 2) == -1  # ffn/p = 96
    a, s = T.mxfp4_empty(130, 40, device="cpu")
    assert a.numel() == T.tpmlp_mxfp4_code_bytes(130, 40) and s.numel() == T.tpmlp_mxfp4_scale_bytes(130, 40)


def quantize(**kw):
    a = dict(X=addr(0), Q=addr(1), S=addr(2), Qt=addr(3), St=addr(4), rows=64, cols=64, ldx=64, p=1, dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_mxfp4_quantize(**a, check=False)


def test_quantize_refusals():
    assert quantize(X=None) == T.ERR_NULL
    assert quantize(S=None) == T.ERR_NULL  # half a pair
    assert quantize(Qt=None) == T.ERR_NULL
    assert quantize(Q=None, S=None, Qt=None, St=None) == T.ERR_NULL
    assert quantize(rows=-1) == T.ERR_SHAPE and quantize(cols=0) == T.ERR_SHAPE and quantize(p=0) == T.ERR_SHAPE
    assert quantize(ldx=32) == T.ERR_SHAPE  # narrower than a row
    assert quantize(rows=1 << 30, cols=1 << 20, ldx=1 << 20) == T.ERR_SHAPE
    assert quantize(p=3) == T.ERR_DIVISIBILITY
    assert quantize(cols=96, p=2) == T.ERR_DIVISIBILITY  # shards of 48 columns: a block would span two
    assert quantize(dt=5) == T.ERR_DTYPE
    assert quantize(Q=addr(1) + 8) == T.ERR_ALIGNMENT
    assert quantize(ldx=68) == T.ERR_ALIGNMENT
    assert quantize(Q=addr(0) + 16) == T.ERR_ALIAS and quantize(St=addr(3) + 16) == T.ERR_ALIAS
    assert quantize() in (T.OK, T.ERR_CUDA, T.ERR_ARCH)


def matmul(**kw):
    a = dict(Aq=addr(0), As=addr(1), Bq=addr(2), Bs=addr(3), bias=None, D=addr(4), m=16, n=64, k=96, out_dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_mxfp4_matmul(**a, check=False)


def test_matmul_and_dequantize_refusals():
    assert matmul(D=None) == T.ERR_NULL and matmul(As=None) == T.ERR_NULL
    assert matmul(m=-1) == T.ERR_SHAPE and matmul(k=0) == T.ERR_SHAPE and matmul(n=0) == T.ERR_SHAPE
    assert matmul(m=1 << 30, n=1 << 20) == T.ERR_SHAPE
    assert matmul(m=(1 << 31) - 100, n=8) == T.ERR_SHAPE and matmul(m=1, n=(1 << 31) - 8) == T.ERR_SHAPE  # within a tile of 2^31
    assert matmul(out_dt=3) == T.ERR_DTYPE
    assert matmul(Bq=addr(2) + 4) == T.ERR_ALIGNMENT
    assert matmul(n=68) == T.ERR_ALIGNMENT and matmul(n=66, out_dt=T.F32) == T.ERR_ALIGNMENT
    assert matmul(D=addr(0)) == T.ERR_ALIAS
    assert matmul(Aq=addr(2), As=addr(3)) in (T.OK, T.ERR_CUDA, T.ERR_ARCH)  # inputs may be the same operand
    deq = lambda q, s, o, r=4, k=32, dt=T.BF16: T.tpmlp_mxfp4_dequantize(q, s, o, r, k, dt, 0, check=False)  # noqa: E731
    assert deq(None, addr(1), addr(2)) == T.ERR_NULL
    assert deq(addr(0), addr(1), addr(2), k=0) == T.ERR_SHAPE
    assert deq(addr(0), addr(1), addr(2), dt=9) == T.ERR_DTYPE
    assert deq(addr(0), addr(1), addr(2) + 4) == T.ERR_ALIGNMENT
    assert deq(addr(0), addr(1), addr(0) + 16) == T.ERR_ALIAS


def fwd(**kw):
    a = dict(X=addr(0), Wq=addr(1), Ws=addr(2), bw_sh=None, Bq=addr(3), Bs=addr(4), b2=None, Z=addr(5), H=addr(6), ws=addr(7), s=4, b=2,
             h=64, ffn=512, p=2, z_dt=T.BF16, stream=0)
    a.update(kw)
    return T.tpmlp_mxfp4_swiglu_mlp_fwd(**a, check=False)


def bwd(**kw):
    a = dict(X=addr(0), Wq=addr(1), Ws=addr(2), Bq=addr(3), Bs=addr(4), H=addr(5), dZ=addr(6), dX=addr(7), dW_sh=addr(8), dB_sh=addr(9),
             dbw_sh=None, db2=None, ws=addr(10), s=4, b=2, h=64, ffn=512, p=2, dx_dt=T.BF16, grad_dt=T.F32, stream=0)
    a.update(kw)
    return T.tpmlp_mxfp4_swiglu_mlp_bwd(**a, check=False)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_block_refusals(call):
    n0 = T.tpmlp_launch_count()
    assert call(X=None) == T.ERR_NULL and call(ws=None) == T.ERR_NULL and call(Ws=None) == T.ERR_NULL
    assert call(h=0) == T.ERR_SHAPE and call(s=-1) == T.ERR_SHAPE and call(p=0) == T.ERR_SHAPE
    assert call(s=1 << 20, b=1 << 12) == T.ERR_SHAPE
    assert call(s=1, b=1, h=8, ffn=1 << 29, p=1) == T.ERR_SHAPE
    assert call(ffn=510, p=4) == T.ERR_DIVISIBILITY and call(ffn=512, p=8, h=64) == T.ERR_DIVISIBILITY  # shards of 64 features
    assert call(h=66, p=4) == T.ERR_DIVISIBILITY
    assert call(**{"z_dt" if call is fwd else "dx_dt": 4}) == T.ERR_DTYPE
    assert call(X=addr(0) + 2) == T.ERR_ALIGNMENT and call(ws=addr(20) + 8) == T.ERR_ALIGNMENT
    assert call(h=60) == T.ERR_ALIGNMENT
    assert call(ws=addr(0)) == T.ERR_ALIAS
    assert call(**{"Z" if call is fwd else "dX": addr(1)}) == T.ERR_ALIAS
    assert T.tpmlp_launch_count() == n0
    assert call(s=0) in (T.OK, T.ERR_CUDA, T.ERR_ARCH)


def test_mode_control():
    for bad in (-1, 6):
        assert T.tpmlp_set_mxfp4_mode(bad, check=False) == T.ERR_SHAPE
    for m in (1, 2, 3, 4, 5, 0):
        assert T.tpmlp_set_mxfp4_mode(m) == T.OK and T.tpmlp_get_mxfp4_mode() == m


def test_reference_rounding():
    """The reference itself: ties to the even code, saturation, the scale of a block, padding."""
    x = np.zeros((1, 40))
    x[0, :10] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -5]
    assert np.array_equal(R.q(x)[0, :10], [4, 0, 1, 1, 2, 2, 4, 4, 6, -4])
    assert not R.q(x)[0, 10:].any()
    assert np.array_equal(R.q(x * 2.0 ** -100), R.q(x) * 2.0 ** -100)
    codes, scales = R.quantize(x)
    assert codes.shape == (1, 32) and scales.tolist() == [[127, 0]]
    t = R.tile_scales(np.arange(256 * 8).reshape(256, 8) % 251, 256, 256)
    assert np.array_equal(R.untile_scales(t, 256, 256), np.arange(256 * 8).reshape(256, 8) % 251)


def test_gradient_formula_against_differences():
    """The backward's formulas with the rounding left out are the derivatives of the block's loss <Z, dZ>:
    central differences in 64 bits.  Truncation about step^2 = 1e-10 and cancellation about 1e-16 / 1e-5 = 1e-11
    of the loss's scale, held to 1e-7."""
    rng = np.random.default_rng(0)
    M, h, f = 5, 8, 128
    same = lambda v: v  # noqa: E731
    x, w, b = rng.standard_normal((M, h)), rng.standard_normal((h, 2 * f)) * 0.3, rng.standard_normal((f, h)) * 0.1
    bw, b2, dz = rng.standard_normal(2 * f) * 0.1, rng.standard_normal(h), rng.standard_normal((M, h))
    loss = lambda x, w, b, bw, b2: float((R.block_fwd(x, w.T, b.T, bw, b2, same)[0] * dz).sum())  # noqa: E731
    args = [x, w, b, bw, b2]
    grads = R.block_bwd(x, w, b, R.block_fwd(x, w.T, b.T, bw, b2, same)[1], dz, same)
    for i, g in enumerate(grads):
        d = rng.standard_normal(args[i].shape)
        at = lambda t: loss(*(a + t * d if j == i else a for j, a in enumerate(args)))  # noqa: E731
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(diff - float((g * d).sum())) <= 1e-7 * max(1.0, abs(diff)), i
