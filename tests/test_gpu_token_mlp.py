"""Joins, layers, the loss and the step as one program: examples/token_mlp.py (GPU).

Gradients against float64, tolerances counted in roundings to bf16: one is relatively off by
at most 2^-8, with a root mean square of less than 2^-9 over a tensor (a value's last place is
worth 2^-8 to 2^-7 of it, and errors spread evenly over half of that, 0.29 of 2^-8 to 2^-7). The
norm's and the activation's slopes are near 1 at these sizes and weights.
"""
import importlib.util
import os

import numpy as np
import pytest

from oracle import adam8
from tests.helpers import log, rel

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_mlp.py")
    spec = importlib.util.spec_from_file_location("token_mlp_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _ids(seed, vocab, rows):
    import torch
    r = np.random.default_rng(seed)
    prev, last, target = torch.from_numpy(r.integers(0, vocab, (3, rows)))
    target[::7] = -1  # padded places
    return prev, last, target


def _loss64(p, blocks, prev, last, target, eps=1e-5):
    """The program's formula on float64 parameters: (loss, log probabilities)."""
    import torch

    def rms(z, gamma):
        return z * torch.rsqrt((z * z).mean(1, keepdim=True) + eps) * gamma

    x = p["last"][last] + p["previous"][prev]
    h = rms(x, p["norm0"])
    for i in range(blocks):
        a = torch.nn.functional.gelu(h @ p[f"w1.{i}"].T + p[f"b1.{i}"], approximate="tanh")
        b = a @ p[f"w2.{i}"].T + p[f"b2.{i}"]
        x = x + p[f"gate{i}"] * rms(b, p[f"post{i}"])
        h = rms(x, p[f"norm{i + 1}"])
    lp = torch.log_softmax(h @ p["head"].T, 1)
    lp = torch.where(target >= 0, lp.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    return -lp.sum() / max(1, int((target >= 0).sum())), lp


def _params64(model):
    return {k: v.detach().double().cpu().requires_grad_() for k, v in model.params.items()}


@pytest.mark.parametrize("vocab,width,hidden,blocks,rows",
                         [(1003, 96, 320, 2, 150), (64, 8, 16, 0, 5), (300, 40, 64, 1, 1),
                          (5000, 256, 512, 1, 700)])
def test_gradients(gpu_lib, vocab, width, hidden, blocks, rows):
    log(f"token mlp gradients {vocab} {width} {hidden} {blocks} {rows}")
    import torch
    model = _example().TokenMlp(vocab, width, hidden, blocks, seed=3)
    prev, last, target = _ids(1, vocab, rows)
    if rows == 1:
        target[0] = 17
    lp, g = model.gradients(prev.cuda(), last.cuda(), target.cuda())
    p = _params64(model)
    loss, want = _loss64(p, blocks, prev, last, target)
    loss.backward()
    # a logit is a sum over a row of h; h, its rounding and the logit's own
    forward = 2 + 3 * blocks
    assert np.abs(lp.cpu().numpy() - want.detach().numpy()).max() < forward * 2.0 ** -8 * 4
    assert set(g) == set(model.params)
    # roundings on the longest path: forward, the logits' gradient, dh, and three a block and back
    roundings = forward + 2 + 3 * blocks + 1
    for k, v in g.items():
        assert v.dtype == torch.float32 and rel(v.double().cpu().numpy(), p[k].grad.numpy()) \
            < roundings * 2.0 ** -9, k
    # the formula's gradient by differences of the loss, along a random direction
    r = torch.Generator().manual_seed(4)
    d = {k: torch.randn(v.shape, generator=r, dtype=torch.float64) for k, v in p.items()}
    with torch.no_grad():
        step = 1e-5
        up, down = [_loss64({k: v + s * step * d[k] for k, v in p.items()}, blocks, prev, last,
                            target)[0] for s in (1, -1)]
        slope = sum((p[k].grad * d[k]).sum() for k in p)
    assert abs((up - down) / (2 * step) - slope) < 1e-6 * (1 + abs(slope))


def test_step(gpu_lib):
    """One call steps vectors as adamw_step does and matrices as the 8-bit oracle does."""
    log("token mlp step")
    import torch
    model = _example().TokenMlp(203, 64, 96, 1, seed=5)
    prev, last, target = (i.cuda() for i in _ids(2, 203, 90))
    for t in (1, 2):
        _, g = model.gradients(prev, last, target)
        before = {k: [s.clone() for s in (model.params[k], *model.adam[k])] for k in model.params}
        model.step(g, t, 1e-2, weight_decay=0.1)
        for k in model.vectors:
            w, m, v = before[k]
            gpu_lib.adamw_step(w, g[k], m, v, t, lr=1e-2)
            assert all(torch.equal(x, y) for x, y in zip((w, m, v), (model.params[k], *model.adam[k])))
        for k in model.matrices:
            w, mc, ms, vc, vs = [s.double().cpu().numpy().ravel() if s.is_floating_point()
                                 else s.cpu().numpy().ravel() for s in before[k]]
            gk = g[k].double().cpu().numpy().ravel()
            m = 0.9 * adam8.decode(mc, ms, "m") + 0.1 * gk
            v = 0.95 * adam8.decode(vc, vs, "v") ** 2 + 0.05 * gk * gk
            over = (1 - 0.9 ** t) * (np.sqrt(v / (1 - 0.95 ** t)) + 1e-8)
            want = w - 1e-2 * (0.1 * w + m / over)
            got = model.params[k].double().cpu().numpy().ravel()
            # the result's rounding to bf16 and, in units of half a step of fp32, 27 for the update
            # (of the terms that its m is the sum of) and 2 for the weight
            m_terms = np.abs(0.9 * adam8.decode(mc, ms, "m")) + np.abs(0.1 * gk)
            f32 = (27e-2 * m_terms / over + 2 * np.abs(w)) * 2.0 ** -24
            assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + 1.01 * f32).all(), k


def test_captured(gpu_lib):
    """Forward, loss and backward in one graph, replayed between eager passes with other rows and
    targets in the same places: bit for bit what the eager passes give."""
    log("token mlp captured")
    import torch
    model = _example().TokenMlp(1003, 96, 320, 2, seed=3)
    sets = []
    for k in range(3):
        prev, last, target = (i.cuda() for i in _ids(10 + k, 1003, 150))
        sets.append((*model.embed(prev, last), target, torch.rand(150, device="cuda")))

    def run(x, b, target, weight):
        logits, saved = model.forward(x, b)
        lp, d = gpu_lib.token_loss(logits, target, weight, out=logits)
        rows, g = model.backward(d, saved)
        return [lp, d, *rows, *(g[k] for k in sorted(g))]

    held = [t.clone() for t in sets[0]]
    run(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*held)
    for k in (1, 0, 2, 1):
        for h, t in zip(held, sets[k]):
            h.copy_(t)
        graph.replay()
        got = [t.clone() for t in out]
        want = run(*sets[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, out):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_example_runs(gpu_lib):
    """Training, scoring and one token at a time: finite values, tokens of the vocabulary, the
    alternatives' best the one that is taken."""
    log("token mlp example")
    import torch
    ex = _example()
    model, losses = ex.train(101, 64, 128, 1, 256, 3)
    assert len(losses) == 3 and np.isfinite(losses).all()
    prev, last, target = (i.cuda() for i in _ids(7, 101, 3))
    s = model.score(prev, last, target, top=4)
    assert s.top_ids.shape == (3, 4) and torch.isfinite(s.top_logprobs).all()
    text = model.generate(prev, last, 5)
    assert text.shape == (3, 5) and ((text >= 0) & (text < 101)).all()
    assert torch.equal(text[:, 0], s.top_ids[:, 0])
