"""The gated feed-forward block with 4-bit operands, trained and served: an example of the MXFP4 entry points.

``GatedMLP`` keeps bf16 weights in the tensor-parallel shard layout (``tpmlp_swiglu_pack``), lays them out as
MXFP4 operands once for each direction they are used in (``tpmlp_mxfp4_quantize``: one read gives both), and runs
the block's forward and backward on them.  Everything is computed by the library; PyTorch holds the memory.

    python -m megatron_tensor_mlp_gb300.mxfp4_block

trains a block towards another one's outputs for a few steps of gradient descent on fp32 master weights, then
serves single tokens with the trained 4-bit weights and compares them with the batch's rows.
"""
from __future__ import annotations

import torch

from . import tpmlp as T


class GatedMLP:
    """Z = (silu(X G + bg) * (X U + bu)) B + b2 with X, the activation and all weights rounded to MXFP4."""

    def __init__(self, gate, up, down, bias_gate=None, bias_up=None, bias_down=None, p: int = 1):
        """gate, up [h, ffn], down [ffn, h] and the biases: bf16 on the GPU.  p: tensor-parallel shards."""
        self.h, self.ffn, self.p = gate.shape[0], gate.shape[-1], p
        h, f = self.h, self.ffn
        self.device = gate.device
        self._check_weights(gate, up, down, bias_gate, bias_up, bias_down)
        self.W = torch.empty((p, h, 2 * f // p), dtype=torch.bfloat16, device=gate.device)
        self.B = torch.empty((f, h), dtype=torch.bfloat16, device=gate.device)
        self.bw = self.b2 = None
        # W as the operand of X W and of dH W^T, B as that of Y B and of dZ B^T
        self.Wt, self.Wn = T.mxfp4_empty(2 * f, h), T.mxfp4_empty(h, 2 * f)
        self.Bt, self.Bn = T.mxfp4_empty(h, f), T.mxfp4_empty(f, h)
        self.load(gate, up, down, bias_gate, bias_up, bias_down)

    def load(self, gate, up, down, bias_gate=None, bias_up=None, bias_down=None):
        """Takes new weights (bf16) and lays out their MXFP4 operands for both directions; biases where given."""
        h, f, p = self.h, self.ffn, self.p
        self._check_weights(gate, up, down, bias_gate, bias_up, bias_down)
        T.tpmlp_swiglu_pack(gate, up, self.W, h, f, p)
        self.B.copy_(down)
        T.tpmlp_mxfp4_quantize(self.W, *self.Wn, *self.Wt, h, 2 * f, 2 * f // p, p)
        T.tpmlp_mxfp4_quantize(self.B, *self.Bn, *self.Bt, f, h, h)
        if bias_gate is not None:
            self.bw = torch.empty(2 * f, dtype=torch.bfloat16, device=gate.device)
            T.tpmlp_swiglu_pack(bias_gate, bias_up, self.bw, 1, f, p)
        if bias_down is not None:
            self.b2 = bias_down

    def _check(self, name, t, *shape):
        """The entry points take addresses: a tensor of another form would be read as if it were this one."""
        if tuple(t.shape) != shape or t.dtype != torch.bfloat16 or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor {list(shape)} on {self.device}, not {t.dtype} {list(t.shape)} "
                             f"with strides {list(t.stride())} on {t.device}")

    def _check_weights(self, gate, up, down, bias_gate, bias_up, bias_down):
        h, f = self.h, self.ffn
        self._check("gate", gate, h, f)
        self._check("up", up, h, f)
        if tuple(down.shape) != (f, h):  # (copied, whatever its type and strides)
            raise ValueError(f"down must be [{f}, {h}], not {list(down.shape)}")
        if (bias_gate is None) != (bias_up is None):
            raise ValueError("bias_gate and bias_up come together")
        for name, b, n in (("bias_gate", bias_gate, f), ("bias_up", bias_up, f), ("bias_down", bias_down, h)):
            if b is not None:
                self._check(name, b, n)

    def _workspace(self, tokens, backward):
        """Scratch of one call.  Each call has its own: two calls on different streams, or from different threads, may run
        at the same time.  (The allocator reuses the memory behind this stream's work only, and costs about a microsecond.)"""
        n = T.tpmlp_mxfp4_swiglu_ws_bytes(tokens, 1, self.h, self.ffn, self.p, backward)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)  # (a shape that is refused gives -1)

    def forward(self, X, save: bool = False):
        """X [tokens, h] bf16 -> Z; with save also the pre-activations that backward needs."""
        m = X.shape[0]
        self._check("X", X, m, self.h)
        Z = torch.empty_like(X)
        H = torch.empty((m, 2 * self.ffn), dtype=torch.bfloat16, device=X.device) if save else None
        if m > 0:  # (an empty tensor has no address to pass)
            T.tpmlp_mxfp4_swiglu_mlp_fwd(X, *self.Wt, self.bw, *self.Bt, self.b2, Z, H, self._workspace(m, 0), m, 1, self.h,
                                         self.ffn, self.p)
        return (Z, H) if save else Z

    def backward(self, X, H, dZ):
        """The gradients of X (bf16) and, fp32, of gate, up, down and, in this order, of the biases that the block has."""
        m, h, f, p = X.shape[0], self.h, self.ffn, self.p
        self._check("X", X, m, h)
        self._check("H", H, m, 2 * f)
        self._check("dZ", dZ, m, h)
        if m == 0:  # (an empty tensor has no address to pass)
            shapes = [(h, f), (h, f), (f, h)] + ([] if self.bw is None else [(f,), (f,)]) + ([] if self.b2 is None else [(h,)])
            return torch.empty_like(X), *(torch.zeros(s, device=X.device) for s in shapes)
        dX = torch.empty_like(X)
        dW, dB = torch.empty((p, h, 2 * f // p), device=X.device), torch.empty((f, h), device=X.device)
        dbw = None if self.bw is None else torch.empty(2 * f, device=X.device)
        db2 = None if self.b2 is None else torch.empty(h, device=X.device)
        T.tpmlp_mxfp4_swiglu_mlp_bwd(X, *self.Wn, *self.Bn, H, dZ, dX, dW, dB, dbw, db2, self._workspace(m, 1), m, 1, h, f, p)
        grads = (dX, *self._unpack(dW, h), dB)
        if dbw is not None:
            grads += tuple(v.view(f) for v in self._unpack(dbw, 1))
        return grads if db2 is None else (*grads, db2)

    def _unpack(self, packed, rows):
        """The gate and up halves [rows, ffn] of an fp32 tensor in the shard layout."""
        G, U = (torch.empty((rows, self.ffn), device=packed.device) for _ in range(2))
        T.tpmlp_swiglu_pack(G, U, packed, rows, self.ffn, self.p, T.F32, inverse=1)
        return G, U


def train_and_serve(tokens=512, h=256, ffn=1024, p=2, steps=40, lr=0.5, seed=0, log=None):
    """Trains a block towards another one's outputs; returns the losses, and the outputs of the first tokens served
    one by one beside the batch's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    teacher = GatedMLP(*(normal(*s).mul_(s[0] ** -0.5).to(bf) for s in ((h, ffn), (h, ffn), (ffn, h))), p=p)
    masters = [normal(*s).mul_(s[0] ** -0.5) for s in ((h, ffn), (h, ffn), (ffn, h))]
    block = GatedMLP(*(w.to(bf) for w in masters), p=p)
    X = normal(tokens, h).to(bf)
    target = teacher.forward(X).float()
    losses = []
    for step in range(steps):
        Z, H = block.forward(X, save=True)
        err = Z.float() - target
        losses.append(float(err.square().mean()))
        if log and step % 10 == 0:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
        _, *grads = block.backward(X, H, (err / tokens).to(bf))
        for w, d in zip(masters, grads):
            w.add_(d, alpha=-lr)
        block.load(*(w.to(bf) for w in masters))
    batch = block.forward(X)
    served = torch.cat([block.forward(X[i:i + 1]) for i in range(8)])
    T.tpmlp_device_status()
    if log:
        log(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; served tokens differ from the batch's by "
            f"{float((served.float() - batch[:8].float()).abs().max()):.2e} at most")
    return losses, served, batch[:8]


if __name__ == "__main__":
    train_and_serve(log=print)
