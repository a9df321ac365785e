"""The example block (mxfp4_block.GatedMLP) on the GPU."""
import numpy as np
import pytest

import gpu_util as U
import mxfp4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Block():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_mlp_gb300 import mxfp4_block
    return mxfp4_block.GatedMLP


def normal(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def make(Block, h, f, seed=0, **kw):
    return Block(normal(seed, h, f, scale=h ** -0.5), normal(seed + 1, h, f, scale=h ** -0.5), normal(seed + 2, f, h, scale=f ** -0.5), **kw)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def test_two_streams_use_one_block(Block):
    """Forwards and backwards of one object on two streams at a time give what each gives alone."""
    import torch
    m = make(Block, 512, 2048)
    X = [normal(10 + i, 700 + 400 * i, 512) for i in range(2)]
    dZ = [normal(20 + i, 700 + 400 * i, 512) for i in range(2)]

    def both(i):
        Z, H = m.forward(X[i], save=True)
        return [Z, H, *m.backward(X[i], H, dZ[i])]

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(outs, want[i]))


def test_no_tokens(Block):
    m = make(Block, 256, 512)
    X = normal(3, 4, 256)[:0]
    Z, H = m.forward(X, save=True)
    grads = m.backward(X, H, X)
    assert Z.shape == (0, 256) and H.shape == (0, 1024) and grads[0].shape == (0, 256)
    assert all(not bool(g.any()) for g in grads[1:])


@pytest.mark.parametrize("p", [1, 2])
def test_gradients_with_biases(Block, p):
    """All gradients of a block with biases against the 64-bit reference; the biases' are used in a step of descent."""
    import torch
    h, f, m = 256, 512, 150
    bias = dict(bias_gate=normal(6, f, scale=0.3), bias_up=normal(7, f, scale=0.3), bias_down=normal(8, h, scale=0.3))
    blk = make(Block, h, f, p=p, **bias)
    X, dZ = normal(4, m, h), normal(5, m, h)
    Z, H = blk.forward(X, save=True)
    dX, dG, dU, dB, dbg, dbu, db2 = blk.backward(X, H, dZ)
    w = host(blk.W.transpose(0, 1).reshape(h, 2 * f))
    packed = R.join(host(bias["bias_gate"])[None], host(bias["bias_up"])[None])[0]
    Zr, Hr = R.block_fwd(host(X), R.q(w.T), R.q(host(blk.B).T), packed, host(bias["bias_down"]))
    U.assert_close(host(Z), Zr, "bf16", "Z")
    ref = R.block_bwd(host(X), R.q(w), R.q(host(blk.B)), host(H), host(dZ))
    for name, got, want in (("dX", dX, ref[0]), ("dB", dB, ref[2]), ("db2", db2, ref[4])):
        U.assert_close(host(got), want, "bf16", name)
    for name, got, want in zip(("dG", "dU"), (dG, dU), R.split(ref[1])):
        U.assert_close(host(got), want, "bf16", name)
    for name, got, want in zip(("dbg", "dbu"), (dbg, dbu), R.split(ref[3][None])):
        U.assert_close(host(got)[None], want, "bf16", name)
    weights = (normal(0, h, f, scale=h ** -0.5), normal(1, h, f, scale=h ** -0.5), normal(2, f, h, scale=f ** -0.5))
    loss = lambda: float((blk.forward(X).double() * dZ.double()).sum())  # noqa: E731
    before = loss()
    step = {k: (v.float() - 0.01 * g).to(torch.bfloat16) for (k, v), g in zip(bias.items(), (dbg, dbu, db2))}
    blk.load(*weights, **step)
    assert loss() < before
