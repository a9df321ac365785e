"""The example block's own part (buffers, checks, what it passes on) with the library's calls recorded instead of made
(CPU only)."""
import pytest
import torch

from megatron_tensor_mlp_gb300 import build as B

B.build()
from megatron_tensor_mlp_gb300 import mxfp4_block  # noqa: E402
from megatron_tensor_mlp_gb300 import tpmlp as T  # noqa: E402

H, F = 64, 256


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, arguments); the arguments are kept, so no buffer is handed out twice meanwhile."""
    made = []
    for name in ("tpmlp_swiglu_pack", "tpmlp_mxfp4_quantize", "tpmlp_mxfp4_swiglu_mlp_fwd", "tpmlp_mxfp4_swiglu_mlp_bwd"):
        monkeypatch.setattr(T, name, lambda *a, _name=name, **kw: made.append((_name, a, kw)))
    empty = T.mxfp4_empty
    monkeypatch.setattr(T, "mxfp4_empty", lambda rows, k, device=None: empty(rows, k, device="cpu"))
    return made


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def block(**kw):
    return mxfp4_block.GatedMLP(bf16(H, F), bf16(H, F), bf16(F, H), **kw)


def of(calls, name):
    return [a for n, a, _ in calls if n == name]


def test_every_call_has_a_workspace_of_its_own(calls):
    """Calls that may run at the same time, on several streams or from several threads, share no scratch."""
    m = block()
    X = bf16(5, H)
    for _ in range(3):
        Z, Hs = m.forward(X, save=True)
        m.backward(X, Hs, X)
    spaces = [a[9] for a in of(calls, "tpmlp_mxfp4_swiglu_mlp_fwd")] + [a[12] for a in of(calls, "tpmlp_mxfp4_swiglu_mlp_bwd")]
    assert len(spaces) == 6
    assert [s.numel() for s in spaces] == ([T.tpmlp_mxfp4_swiglu_ws_bytes(5, 1, H, F, 1, 0)] * 3
                                           + [T.tpmlp_mxfp4_swiglu_ws_bytes(5, 1, H, F, 1, 1)] * 3)
    assert len({s.data_ptr() for s in spaces}) == 6


def test_no_tokens(calls):
    """An empty batch is a batch: no output rows, gradients of zero, nothing launched (an empty tensor's address is NULL,
    which the entry points refuse)."""
    m = block()
    del calls[:]
    X = bf16(0, H)
    Z, Hs = m.forward(X, save=True)
    assert Z.shape == (0, H) and Hs.shape == (0, 2 * F) and m.forward(X).shape == (0, H)
    dX, dG, dU, dB = m.backward(X, Hs, X)
    assert not calls
    assert dX.shape == (0, H) and dX.dtype == torch.bfloat16
    for d, shape in ((dG, (H, F)), (dU, (H, F)), (dB, (F, H))):
        assert d.shape == shape and d.dtype == torch.float32 and not d.any()
