"""A pre-norm MLP block trained with this library alone: y = x + W2 gelu(W1 norm(x) + b1) + b2.

The layer operators run the block forward and backward, FOAM steps its two
weight matrices and AdamW its vectors. With ``keep="int8"`` or ``"e4m3"`` the
activations the backward pass needs (the block's input, the norm's output and
the pre-activation) are kept in 8 bits: at 1536 and 6144, 0.31 of the bytes of a
block that keeps those three and the activation's output in bf16; the activation
is recomputed from the pre-activation.

    python examples/mlp_block.py [--width 1536] [--hidden 6144] [--tokens 4096]
                                 [--steps 20] [--keep int8|e4m3|none]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_aware_optimizers_amd as mao  # noqa: E402

ACT = "gelu_tanh"


def _foam_state(w):
    m, n = w.shape
    f32 = dict(dtype=torch.float32, device=w.device)
    return {"M": torch.zeros((m, n), **f32), "R": torch.zeros((n, n), **f32),
            "QR": torch.eye(n, **f32), "r": torch.zeros(m, **f32), "c": torch.zeros(n, **f32),
            "aux": torch.zeros(4, **f32)}


class MlpBlock:
    """Weights (bf16 matrices, fp32 vectors) and optimizer state of one block;
    ``width`` and ``hidden`` multiples of 8."""

    def __init__(self, width, hidden, keep="int8", device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g).to(device)

        self.keep = keep
        self.matrices = {"w1": (0.5 * normal(hidden, width) / width ** 0.5).bfloat16(),
                         "w2": (0.5 * normal(width, hidden) / hidden ** 0.5).bfloat16()}
        self.vectors = {"b1": torch.zeros(hidden, device=device),
                        "b2": torch.zeros(width, device=device),
                        "gamma": torch.ones(width, device=device),
                        "beta": torch.zeros(width, device=device)}
        self.foam = {k: _foam_state(w) for k, w in self.matrices.items()}
        self.adam = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.vectors.items()}

    def _kept(self, x):
        return x if self.keep == "none" else mao.q8_quantize(x, self.keep)

    def forward(self, x):
        """(y, what the backward pass needs)"""
        v = self.vectors
        h, mean, rstd = mao.layer_norm(x, v["gamma"], v["beta"])
        z = torch.empty((x.shape[0], self.matrices["w1"].shape[0]), dtype=x.dtype, device=x.device)
        a = mao.linear(h, self.matrices["w1"], v["b1"], act=ACT, preact=z)
        y = mao.linear(a, self.matrices["w2"], v["b2"], residual=x)
        return y, (self._kept(x), self._kept(h), self._kept(z), mean, rstd)

    def backward(self, dy, saved):
        """(dx, gradients by name)"""
        x, h, z, mean, rstd = saved
        g = {}
        g["w2"], g["b2"] = mao.linear_backward_weight(dy, z, x_act=ACT)
        dz = mao.linear_backward_input(dy, self.matrices["w2"], act=ACT, preact=z)
        g["w1"], g["b1"] = mao.linear_backward_weight(dz, h)
        dh = mao.linear_backward_input(dz, self.matrices["w1"])
        dx, g["gamma"], g["beta"] = mao.layer_norm_backward(dh, x, self.vectors["gamma"], mean,
                                                            rstd, add=dy)
        return dx, g

    def step(self, grads, t, lr):
        for k, w in self.matrices.items():
            mao.foam_step(w, grads[k], self.foam[k], t, lr=lr, fwd_rot="bf16x3",
                          refresh_prod="bf16x3", back_rot_dtype="bf16")
        for k, v in self.vectors.items():
            mao.adamw_step(v, grads[k], *self.adam[k], t, lr=lr)


def train(width, hidden, tokens, steps, keep, lr=2e-3, seed=0, device="cuda"):
    """Losses of a block that learns another, fixed block's outputs."""
    block = MlpBlock(width, hidden, keep, device, seed)
    teacher = MlpBlock(width, hidden, "none", device, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    x = torch.randn((tokens, width), generator=g).to(device).bfloat16()
    target = teacher.forward(x)[0].float()
    losses = []
    for t in range(1, steps + 1):
        y, saved = block.forward(x)
        diff = y.float() - target
        losses.append(float((diff * diff).mean()))
        _, grads = block.backward((diff * (2.0 / diff.numel())).bfloat16(), saved)
        block.step(grads, t, lr)
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--width", type=int, default=1536)
    p.add_argument("--hidden", type=int, default=6144)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--keep", choices=["int8", "e4m3", "none"], default="int8")
    a = p.parse_args()
    for i, loss in enumerate(train(a.width, a.hidden, a.tokens, a.steps, a.keep), 1):
        print(f"step {i:3d}  loss {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
