"""A mixture-of-experts feed-forward layer on the library's entry points: an example, trained and served.

``ExpertLayer`` normalises its input (``tpmlp_layernorm_fwd``), takes router logits from the column layer
(``tpmlp_column_fwd`` without activation), routes (``tpmlp_moe_route``), runs the gated experts on the rows that the
routing made (``tpmlp_moe_matmul``) and combines their rows into tokens (``tpmlp_moe_combine``); its backward walks the
same way back.  The plan of rows stays on the device: nothing is read back on the way.  PyTorch holds the memory.

    python -m megatron_tensor_mlp_gb300.moe_block

trains a layer towards another one's outputs for a few steps of gradient descent on fp32 master weights, then serves
single tokens with the trained weights and compares them with the batch's rows.
"""
from __future__ import annotations

import torch

from . import tpmlp as T

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class ExpertLayer:
    """z[t] = sum_j w[t, j] E_j(LN(x[t])) over the k experts with the largest logits LN(x) R, w their softmax;
    E(v) = (silu(v G) * (v U)) D."""

    def __init__(self, gamma, beta, router, gate, up, down, k: int):
        """gamma, beta [h], router [h, experts], gate, up [experts, h, ffn], down [experts, ffn, h]: contiguous bf16 on the GPU.
        experts a multiple of 8, ffn of 128."""
        self.experts, self.h, self.ffn = gate.shape
        self.k, self.device = k, gate.device
        if self.device.type != "cuda":
            raise ValueError(f"the weights must be on a GPU, not on {self.device}")
        self.W1 = torch.empty((self.experts, self.h, 2 * self.ffn), dtype=BF, device=self.device)
        self.load(gamma, beta, router, gate, up, down)

    def load(self, gamma, beta, router, gate, up, down):
        """Takes new weights; gate and up are packed into the first layer's columns."""
        e, h, f = self.experts, self.h, self.ffn
        for name, t, shape in (("gamma", gamma, (h,)), ("beta", beta, (h,)), ("router", router, (h, e)), ("gate", gate, (e, h, f)),
                               ("up", up, (e, h, f)), ("down", down, (e, f, h))):
            self._check(name, t, *shape)
        self.gamma, self.beta, self.router, self.W2 = gamma, beta, router, down
        with torch.cuda.device(self.device):  # (calls go to the current device)
            T.tpmlp_swiglu_pack(gate, up, self.W1, e * h, f, 1)

    def _check(self, name, t, *shape):
        """The entry points take addresses: a tensor of another form would be read as if it were this one."""
        if tuple(t.shape) != shape or t.dtype != BF or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor {list(shape)} on {self.device}, not {t.dtype} {list(t.shape)} "
                             f"with strides {list(t.stride())} on {t.device}")

    def _new(self, *shape, dtype=BF):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def forward(self, X, save: bool = False):
        """X [tokens, h] bf16 -> Z; with save also what backward needs."""
        t, h, f, e, k = X.shape[0], self.h, self.ffn, self.experts, self.k
        self._check("X", X, t, h)
        n, mean, rstd = self._new(t, h), self._new(t, dtype=F32), self._new(t, dtype=F32)
        logits, ids, w = self._new(t, e), self._new(t, k, dtype=I32), self._new(t, k, dtype=F32)
        offsets, row_token, slot_row = self._new(e + 1, dtype=I32), self._new(t * k, dtype=I32), self._new(t, k, dtype=I32)
        Z, Y, O = self._new(t, h), self._new(t * k, f), self._new(t * k, h)  # noqa: E741
        H = self._new(t * k, 2 * f, dtype=F32) if save else None
        out = (Z, (X, n, mean, rstd, logits, ids, w, offsets, row_token, slot_row, Y, O, H)) if save else Z
        if t == 0:  # (an empty tensor has no address to pass)
            return out
        with torch.cuda.device(self.device):
            ws = self._new(T.tpmlp_moe_route_ws_bytes(t, e, k), dtype=torch.uint8)
            T.tpmlp_layernorm_fwd(X, self.gamma, self.beta, n, mean, rstd, t, h, h, h)
            T.tpmlp_column_fwd(n, self.router, None, logits, None, t, 1, h, e, 1, act=T.ACT_NONE)
            T.tpmlp_moe_route(logits, ids, w, offsets, row_token, slot_row, ws, t, e, k)
            T.tpmlp_moe_matmul(n, row_token, offsets, self.W1, None, Y, H, t, t * k, e, h, 2 * f, act=T.ACT_SWIGLU_H32)
            T.tpmlp_moe_matmul(Y, None, offsets, self.W2, None, O, None, t * k, t * k, e, f, h)
            T.tpmlp_moe_combine(O, slot_row, w, Z, t, t * k, k, h)
        return out

    def backward(self, saved, dZ):
        """The gradients of X (bf16) and, fp32, of gamma, beta, router, gate, up and down."""
        X, n, mean, rstd, logits, ids, w, offsets, row_token, slot_row, Y, O, H = saved  # noqa: E741
        t, h, f, e, k = X.shape[0], self.h, self.ffn, self.experts, self.k
        self._check("dZ", dZ, t, h)
        r = t * k
        grads = [self._new(h, dtype=F32), self._new(h, dtype=F32), self._new(h, e, dtype=F32)]
        dW1, dW2 = self._new(e, h, 2 * f, dtype=F32), self._new(e, f, h, dtype=F32)
        G, U = self._new(e, h, f, dtype=F32), self._new(e, h, f, dtype=F32)
        dX = self._new(t, h)
        if t == 0:
            return dX, *(g.zero_() for g in (*grads, G, U, dW2))
        dO, dH, dR = self._new(r, h), self._new(r, 2 * f), self._new(r, h)
        dw, dlogits, dn, dn_router = self._new(t, k, dtype=F32), self._new(t, e), self._new(t, h), self._new(t, h)
        ws = self._new(T.tpmlp_layernorm_ws_bytes(t, h), dtype=torch.uint8)
        with torch.cuda.device(self.device):
            T.tpmlp_moe_combine_bwd(O, slot_row, w, dZ, dO, dw, t, r, k, h)
            T.tpmlp_moe_matmul_dx(dO, offsets, self.W2, H, dH, r, e, f, h, act=T.ACT_SWIGLU_H32)
            T.tpmlp_moe_matmul_dw(Y, None, offsets, dO, dW2, None, r, r, e, f, h)
            T.tpmlp_moe_matmul_dx(dH, offsets, self.W1, None, dR, r, e, h, 2 * f)
            T.tpmlp_moe_matmul_dw(n, row_token, offsets, dH, dW1, None, t, r, e, h, 2 * f)
            T.tpmlp_moe_combine(dR, slot_row, None, dn, t, r, k, h)
            T.tpmlp_moe_route_bwd(logits, ids, w, dw, dlogits, t, e, k)
            T.tpmlp_column_bwd(n, self.router, dlogits, dn_router, grads[2], None, t, 1, h, e, 1)
            dn.add_(dn_router)
            T.tpmlp_layernorm_bwd(X, self.gamma, mean, rstd, dn, dX, grads[0], grads[1], ws, t, h, h, h, h)
            T.tpmlp_swiglu_pack(G, U, dW1, e * h, f, 1, T.F32, inverse=1)
        return dX, *grads, G, U, dW2


def train_and_serve(tokens=512, h=256, ffn=256, experts=8, k=2, steps=30, lr=0.5, seed=0, log=None):
    """Trains a layer towards another one's outputs; returns the losses, and the outputs of the first tokens served one by one
    beside the batch's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    shapes = ((h,), (h,), (h, experts), (experts, h, ffn), (experts, h, ffn), (experts, ffn, h))

    def weights():
        return [normal(*s).mul_(0.1 if len(s) == 1 else s[-2] ** -0.5).add_(1 if i == 0 else 0) for i, s in enumerate(shapes)]

    teacher = ExpertLayer(*(w.to(BF) for w in weights()), k)
    masters = weights()
    layer = ExpertLayer(*(w.to(BF) for w in masters), k)
    X = normal(tokens, h).to(BF)
    target = teacher.forward(X).float()
    losses = []
    for step in range(steps):
        Z, saved = layer.forward(X, save=True)
        err = Z.float() - target
        losses.append(float(err.square().mean()))
        if log and step % 10 == 0:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
        _, *grads = layer.backward(saved, (err / tokens).to(BF))
        for w, d in zip(masters, grads):
            w.add_(d, alpha=-lr)
        layer.load(*(w.to(BF) for w in masters))
    batch = layer.forward(X)
    served = torch.cat([layer.forward(X[i:i + 1]) for i in range(8)])
    T.tpmlp_device_status()
    if log:
        log(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; served tokens differ from the batch's by "
            f"{float((served.float() - batch[:8].float()).abs().max()):.2e} at most")
    return losses, served, batch[:8]


if __name__ == "__main__":
    train_and_serve(log=print)
