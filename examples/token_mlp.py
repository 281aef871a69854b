"""A small language model trained with this library alone: the next token from the last two.

The rows of two embeddings (of the last token and of the one before it) are added and normed by
``residual_norm``; each block is an MLP of two ``linear`` layers that joins the residual stream
through a norm of its output, a gate per channel and the next block's norm, ``residual_norm``
again; the head's logits go through ``token_loss``, which leaves their gradient in their place.
``adamw_step_many`` steps everything in one call, the matrices with states in 8 bits. Text is
continued one token at a time with ``token_logprobs``.

    python examples/token_mlp.py [--vocab 5000] [--width 512] [--hidden 2048] [--blocks 2]
                                 [--tokens 8192] [--steps 20]
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


class TokenMlp:
    """Weights (bf16 matrices, fp32 vectors) and AdamW states; ``width`` and ``hidden``
    multiples of 8. The residual stream is fp32, the blocks' inputs and outputs are bf16."""

    def __init__(self, vocab, width, hidden, blocks, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g) / shape[1] ** 0.5).to(device).bfloat16()

        ones = dict(dtype=torch.float32, device=device)
        self.blocks = blocks
        self.matrices = {"last": normal(vocab, width), "previous": normal(vocab, width),
                         "head": normal(vocab, width)}
        self.vectors = {"norm0": torch.ones(width, **ones)}
        for i in range(blocks):
            self.matrices[f"w1.{i}"] = normal(hidden, width)
            self.matrices[f"w2.{i}"] = normal(width, hidden)
            self.vectors[f"b1.{i}"] = torch.zeros(hidden, **ones)
            self.vectors[f"b2.{i}"] = torch.zeros(width, **ones)
            self.vectors[f"post{i}"] = torch.ones(width, **ones)
            self.vectors[f"gate{i}"] = torch.full((width,), 0.5, **ones)
            self.vectors[f"norm{i + 1}"] = torch.ones(width, **ones)
        self.params = {**self.matrices, **self.vectors}
        self.adam = {k: mao.adamw8_state(w) for k, w in self.matrices.items()}
        self.adam.update({k: (torch.zeros_like(v), torch.zeros_like(v))
                          for k, v in self.vectors.items()})

    def embed(self, previous, last):
        """The rows of both embeddings: of the stream (fp32) and of what joins it."""
        return self.matrices["last"][last].float(), self.matrices["previous"][previous]

    def _join(self, i):
        v = self.vectors
        if i == 0:
            return dict(pre_gamma=v["norm0"])
        return dict(gate=v[f"gate{i - 1}"], post="rms", post_gamma=v[f"post{i - 1}"],
                    pre_gamma=v[f"norm{i}"])

    def forward(self, x, b):
        """(logits, what the backward pass needs)"""
        m, v, saved = self.matrices, self.vectors, []
        for i in range(self.blocks + 1):
            x, h, stats = mao.residual_norm(x, b, **self._join(i))
            saved.append([b, x, h, stats])
            if i < self.blocks:
                z = torch.empty((x.shape[0], m[f"w1.{i}"].shape[0]), dtype=h.dtype, device=h.device)
                a = mao.linear(h, m[f"w1.{i}"], v[f"b1.{i}"], act=ACT, preact=z)
                b = mao.linear(a, m[f"w2.{i}"], v[f"b2.{i}"])
                saved[i].append(z)
        return mao.linear(h, m["head"]), saved

    def backward(self, dlogits, saved):
        """(gradients of the embeddings' rows, gradients by name)"""
        m, g, dr = self.matrices, {}, None
        g["head"], _ = mao.linear_backward_weight(dlogits, saved[-1][2], dbias=False)
        dh = mao.linear_backward_input(dlogits, m["head"])
        for i in range(self.blocks, -1, -1):
            if i < self.blocks:
                h, z = saved[i][2], saved[i][4]
                g[f"w2.{i}"], g[f"b2.{i}"] = mao.linear_backward_weight(db, z, x_act=ACT)
                dz = mao.linear_backward_input(db, m[f"w2.{i}"], act=ACT, preact=z)
                g[f"w1.{i}"], g[f"b1.{i}"] = mao.linear_backward_weight(dz, h)
                dh = mao.linear_backward_input(dz, m[f"w1.{i}"])
            b, r, _, stats = saved[i][:4]
            join = mao.residual_norm_backward(dh, dr, b, r, stats, out=dr, **self._join(i))
            dr, db, g[f"norm{i}"] = join.dX, join.dB, join.dpre_gamma
            if i > 0:
                g[f"gate{i - 1}"], g[f"post{i - 1}"] = join.dgate, join.dpost_gamma
        return (dr, db), g

    def gradients(self, previous, last, targets):
        """(log probabilities of the targets, gradients of their mean's negative by name).
        Targets below 0 are not counted."""
        weight = (targets >= 0).float()
        weight /= weight.sum().clamp(min=1)
        logits, saved = self.forward(*self.embed(previous, last))
        logprob, dlogits = mao.token_loss(logits, targets, weight, out=logits)
        (dlast, dprevious), g = self.backward(dlogits, saved)
        for name, ids, rows in (("last", last, dlast), ("previous", previous, dprevious)):
            g[name] = torch.zeros(self.matrices[name].shape, dtype=torch.float32,
                                  device=rows.device)
            g[name].index_put_((ids,), rows.float(), accumulate=True)
        return logprob, g

    def step(self, grads, t, lr, weight_decay=0.01):
        mao.adamw_step_many([(w, grads[k], *self.adam[k]) for k, w in self.params.items()], t, lr=lr,
                            weight_decay=[weight_decay if k in self.matrices else 0.0
                                          for k in self.params])

    def score(self, previous, last, targets, top=0):
        """Log probabilities, entropies and alternatives of given continuations."""
        logits, _ = self.forward(*self.embed(previous, last))
        return mao.token_logprobs(logits, targets, top=top)

    def generate(self, previous, last, count):
        """The most likely continuation: ``count`` tokens for each row, one at a time."""
        out = []
        for _ in range(count):
            previous, last = last, self.score(previous, last, None, top=1).top_ids[:, 0]
            out.append(last)
        return torch.stack(out, dim=1)


def train(vocab, width, hidden, blocks, tokens, steps, lr=2e-3, seed=0, device="cuda"):
    """(model, losses): the next token is the sum of the last two, modulo the vocabulary."""
    model = TokenMlp(vocab, width, hidden, blocks, device, seed)
    g = torch.Generator().manual_seed(seed + 1)
    losses = []
    for t in range(1, steps + 1):
        previous, last = torch.randint(0, vocab, (2, tokens), generator=g).to(device)
        logprob, grads = model.gradients(previous, last, (previous + last) % vocab)
        model.step(grads, t, lr)
        losses.append(-float(logprob.mean()))
    return model, losses


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("vocab", 5000), ("width", 512), ("hidden", 2048), ("blocks", 2),
                          ("tokens", 8192), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    _, losses = train(a.vocab, a.width, a.hidden, a.blocks, a.tokens, a.steps)
    for i, loss in enumerate(losses, 1):
        print(f"step {i:3d}  loss {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
