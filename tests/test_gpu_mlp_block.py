"""The layer operators and the optimizer steps together: examples/mlp_block.py (GPU).

The block's gradients against float64 on the values the block itself holds, and a
short training run with and without 8-bit checkpoints.
"""
import importlib.util
import os

import numpy as np
import pytest

from oracle import layers as ref
from tests.helpers import log, rel
from tests.test_gpu_layers import host, values

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("keep", ["none", "int8", "e4m3"])
def test_block_gradients(gpu_lib, keep):
    import torch
    log(f"mlp block gradients {keep}")
    ex = _example()
    block = ex.MlpBlock(96, 320, keep)
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.standard_normal((150, 96))).to("cuda").bfloat16()
    dy = torch.from_numpy(r.standard_normal((150, 96))).to("cuda").bfloat16()
    y, saved = block.forward(x)
    dx, g = block.backward(dy, saved)
    w1, w2 = host(block.matrices["w1"]), host(block.matrices["w2"])
    v = {k: host(t) for k, t in block.vectors.items()}
    # forward: bf16 roundings of h and a, each 2^-9 of its values on average
    wh, mean, rstd = ref.layer_norm(host(x), v["gamma"], v["beta"], 1e-5)
    wa, wz = ref.linear(wh, w1, v["b1"], "gelu_tanh")
    wy, _ = ref.linear(wa, w2, v["b2"], residual=host(x))
    assert rel(host(y), wy) < 6e-3
    # backward, from what was kept
    kx, kh, kz = [host(s) if keep == "none" else values(s) for s in saved[:3]]
    wdw2, wdb2 = ref.linear_backward_weight(host(dy), kz, "gelu_tanh")
    wdz = ref.linear_backward_input(host(dy), w2, "gelu_tanh", kz)
    wdw1, wdb1 = ref.linear_backward_weight(wdz, kh)
    wdx, wdg, wdb = ref.layer_norm_backward(wdz @ w1, kx, v["gamma"], mean, rstd)
    want = {"w2": wdw2, "b2": wdb2, "w1": wdw1, "b1": wdb1, "gamma": wdg, "beta": wdb}
    for k, w in want.items():
        # at most three bf16 roundings lie between dy and any of these
        assert rel(host(g[k]), w) < 8e-3, (k, rel(host(g[k]), w))
    assert rel(host(dx), wdx + host(dy)) < 8e-3


def test_block_learns_alike_with_8_bit_checkpoints(gpu_lib):
    log("mlp block training")
    ex = _example()
    runs = {k: ex.train(128, 512, 1024, 30, k) for k in ("none", "int8", "e4m3")}
    for k, losses in runs.items():
        assert np.isfinite(losses).all(), k
        assert losses[-1] < 0.5 * losses[0], (k, losses[0], losses[-1])
    # checkpoints change the gradients by well under a percent (int8) or a few (e4m3)
    assert abs(runs["int8"][-1] / runs["none"][-1] - 1) < 0.05
    assert abs(runs["e4m3"][-1] / runs["none"][-1] - 1) < 0.2
