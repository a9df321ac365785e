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


def biases():
    return dict(bias_gate=bf16(F), bias_up=bf16(F), bias_down=bf16(H))


def test_gradients_of_the_biases(calls):
    """A block with biases asks for their gradients and returns them, in the constructor's order."""
    X = bf16(5, H)
    m = block(**biases(), p=2)
    Z, Hs = m.forward(X, save=True)
    grads = m.backward(X, Hs, X)
    dbw, db2 = of(calls, "tpmlp_mxfp4_swiglu_mlp_bwd")[0][10:12]
    assert dbw.numel() == 2 * F and db2.numel() == H and dbw.dtype == db2.dtype == torch.float32
    assert [tuple(g.shape) for g in grads] == [(5, H), (H, F), (H, F), (F, H), (F,), (F,), (H,)]
    assert grads[6].data_ptr() == db2.data_ptr()
    unpack = of(calls, "tpmlp_swiglu_pack")[-1]  # (G, U, packed, rows, ffn, p, ...)
    assert [t.data_ptr() for t in unpack[:3]] == [grads[4].data_ptr(), grads[5].data_ptr(), dbw.data_ptr()] and unpack[3:6] == (1, F, 2)
    assert [tuple(g.shape) for g in m.backward(X[:0], Hs[:0], X[:0])] == [(0, H)] + [tuple(g.shape) for g in grads[1:]]
    # only some of them
    assert len(block(bias_down=bf16(H)).backward(X, Hs, X)) == 5
    assert len(block(bias_gate=bf16(F), bias_up=bf16(F)).backward(X, Hs, X)) == 6
    assert len(block().backward(X, Hs, X)) == 4


def test_new_biases_are_taken(calls):
    m = block(**biases())
    new = biases()
    m.load(bf16(H, F), bf16(H, F), bf16(F, H), **new)
    X = bf16(5, H)
    m.forward(X)
    pack = of(calls, "tpmlp_swiglu_pack")[-1]
    args = of(calls, "tpmlp_mxfp4_swiglu_mlp_fwd")[-1]
    assert pack[0] is new["bias_gate"] and pack[1] is new["bias_up"] and args[3] is pack[2] and args[6] is new["bias_down"]


def test_tensors_of_another_form_are_refused(calls):
    """The entry points take addresses: a tensor of another type, shape or stride would be read as if it were the right
    one, past its end at worst.  Nothing is called with one."""
    m = block(**biases())
    X = bf16(5, H)
    Z, Hs = m.forward(X, save=True)
    good = dict(X=X, H=Hs, dZ=X)
    del calls[:]
    wrong = [X.float(), X.half(), bf16(5, 2 * H)[:, :H], bf16(1, H).expand(5, H), bf16(H, 5).t(), bf16(5, H + 8), bf16(5 * H), bf16(5, 1, H),
             torch.zeros(5, H, dtype=torch.bfloat16, device="meta")]
    for bad in wrong:
        with pytest.raises(ValueError):
            m.forward(bad)
        for name in ("X", "dZ"):
            with pytest.raises(ValueError):
                m.backward(**{**good, name: bad})
    for bad in (bf16(4, 2 * F), Hs.float(), bf16(5, F), bf16(1, 2 * F).expand(5, 2 * F)):
        with pytest.raises(ValueError):
            m.backward(X, bad, X)
    with pytest.raises(ValueError):
        m.backward(X, Hs, bf16(4, H))
    weights = dict(gate=bf16(H, F), up=bf16(H, F), down=bf16(F, H), **biases())
    for name, bad in (("gate", bf16(H, F).float()), ("gate", bf16(F, H).t()), ("up", bf16(H, F + 8)), ("up", bf16(F, H)), ("down", bf16(1, H)),
                      ("bias_gate", torch.zeros(F)), ("bias_up", bf16(F - 8)), ("bias_up", None), ("bias_gate", None),
                      ("bias_down", bf16(2 * H)[::2])):
        with pytest.raises(ValueError):
            m.load(**{**weights, name: bad})
        with pytest.raises(ValueError):
            mxfp4_block.GatedMLP(**{**weights, name: bad})
    assert not calls
    m.forward(X), m.backward(**good), m.load(**weights)
    assert len(of(calls, "tpmlp_mxfp4_swiglu_mlp_fwd")) == len(of(calls, "tpmlp_mxfp4_swiglu_mlp_bwd")) == 1
