"""Refusals of gated experts with fp32 pre-activations (CPU only: ahead of any CUDA call)."""
import pytest

torch = pytest.importorskip("torch")

import test_moe_host as H  # noqa: E402

T = H.T


def test_refusals():
    gated = dict(act=T.ACT_SWIGLU_H32)
    assert H.matmul(**gated, H=H.addr(5)) in H.REACHED and H.matmul(**gated) in H.REACHED
    assert H.matmul(**gated, N=384) == T.ERR_DIVISIBILITY and H.matmul(**gated, out_dt=T.F32) == T.ERR_DTYPE
    assert H.matmul(**gated, H=H.addr(5) + 8) == T.ERR_ALIGNMENT
    assert H.matmul(act=4) == T.ERR_SHAPE
    # 16 rows of 256 values take twice the bytes that bf16 takes
    end = H.addr(3) - 16 * 256 * 2
    assert H.matmul(act=T.ACT_SWIGLU, H=end) in H.REACHED and H.matmul(**gated, H=end) == T.ERR_ALIAS
    assert H.dx(**gated) == T.ERR_NULL and H.dx(**gated, H=H.addr(4)) in H.REACHED
    assert H.dx(**gated, H=H.addr(4), K=192) == T.ERR_DIVISIBILITY and H.dx(**gated, H=H.addr(4), dx_dt=T.F32) == T.ERR_DTYPE
    end = H.addr(3) - 16 * 256 * 2
    assert H.dx(act=T.ACT_SWIGLU, H=end) in H.REACHED and H.dx(**gated, H=end) == T.ERR_ALIAS


def test_the_dense_layers_refuse_it():
    st = T.tpmlp_column_fwd(H.addr(0), H.addr(1), None, H.addr(2), None, 4, 2, 64, 256, 2, act=T.ACT_SWIGLU_H32, stream=0, check=False)
    assert st == T.tpmlp_column_fwd(H.addr(0), H.addr(1), None, H.addr(2), None, 4, 2, 64, 256, 2, act=9, stream=0, check=False) != T.OK
