"""The weight gradient through a recomputed activation, kept in fp32 (GPU).

dW = dY^T act(x) with dY in bf16 and act(x) from a saved bf16 tensor or an 8-bit
checkpoint: an fp32 result has the error of fp32 arithmetic, not of an operand
rounded to bf16. Bound: u = 2^-24, B = 2^-8 as in test_gpu_layers. The activation
is evaluated to 2e-6 of max(1, |x|) and enters the product as two bf16 parts, which
leaves B^2 of it; each part's product adds (K + 8) u of its magnitudes.
"""
import numpy as np
import pytest

from oracle import layers as ref
from tests.helpers import log
from tests.test_gpu_layers import B, U, _kept, _product_bound, check, dev, host

pytestmark = pytest.mark.gpu


def _bound(dy, x, act, first=0.0):
    a = np.abs(ref.act(x, act))
    d = np.abs(dy).T.astype(np.float64)
    rows = dy.shape[0]
    p = _product_bound(dy.T, a * (1 + B), rows)
    return p + d @ (2e-6 * np.maximum(1, np.abs(x)) + B * B * a) + 4 * U * (p / ((rows + 8) * U)
                                                                          + np.abs(first))


# rows, k, n: tiles alone and with K split, one row, a large tile
@pytest.mark.parametrize("act,saved", [("gelu", "int8"), ("gelu_tanh", "bf16"), ("silu", "e4m3"),
                                       ("relu", "bf16")])
@pytest.mark.parametrize("shape", [(1, 40, 17), (130, 100, 257), (999, 70, 33), (77, 1100, 200)])
def test_fp32_result_has_fp32_error(gpu_lib, shape, act, saved):
    log(f"recomputed activation {shape} {act} {saved}")
    rows, k, n = shape
    r = np.random.default_rng(3)
    dy = ref_bf16(r.standard_normal((rows, n)))
    kept, x = _kept(gpu_lib, 2 * r.standard_normal((rows, k)), saved)
    dw, db = gpu_lib.linear_backward_weight(dev(dy, "bf16", 8), kept, x_act=act)
    want, wb = ref.linear_backward_weight(dy, x, act)
    check(dw, want, _bound(dy, x, act), "dw")
    check(db, wb, (rows + 8) * U * np.abs(dy).sum(axis=0) + 1e-30, "dbias")


def ref_bf16(x):
    from synth import bf16_round
    return bf16_round(np.asarray(x, np.float32))


def test_fp32_result_on_large_tiles(gpu_lib):
    import torch
    log("recomputed activation, large tiles")
    rows, k, n = 1300, 2817, 2600
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    dy = torch.randn((rows, n), generator=g, device="cuda").bfloat16()
    x = gpu_lib.padded(torch.randn((rows, k), generator=g, device="cuda").bfloat16())
    dw, _ = gpu_lib.linear_backward_weight(dy, x, x_act="silu")
    d, xd = dy.double(), x.double()
    a = xd * torch.sigmoid(xd)
    dt = d.t().contiguous()
    want = torch.matmul(dt, a)
    mag = torch.matmul(dt.abs(), a.abs() * (1 + B))
    bound = (rows + 12) * U * mag + torch.matmul(
        dt.abs(), 2e-6 * xd.abs().clamp(min=1) + B * B * a.abs())
    err = (dw.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("shape", [(90, 133, 70), (700, 70, 60)])
def test_fp32_result_accumulates(gpu_lib, shape):
    log(f"recomputed activation, accumulated {shape}")
    rows, k, n = shape
    r = np.random.default_rng(9)
    dw = db = None
    want = np.zeros((n, k))
    bound = np.zeros((n, k))
    wb = np.zeros(n)
    for i in range(2):
        dy = ref_bf16(r.standard_normal((rows, n)))
        kept, x = _kept(gpu_lib, r.standard_normal((rows, k)), "int8")
        bound += _bound(dy, x, "gelu", want)
        p, pb = ref.linear_backward_weight(dy, x, "gelu")
        want, wb = want + p, wb + pb
        dw, db = gpu_lib.linear_backward_weight(dev(dy, "bf16"), kept, x_act="gelu", out=dw,
                                                dbias=db, accumulate=i > 0)
    check(dw, want, bound, "dw")
    check(db, wb, 2 * (rows + 12) * U * rows * np.ones(n) * 6, "dbias")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_infinite_activation_stays_infinite(gpu_lib, act):
    import torch
    log(f"recomputed activation, infinity {act}")
    r = np.random.default_rng(5)
    dy = ref_bf16(r.standard_normal((40, 24)))
    x = ref_bf16(r.standard_normal((40, 56)))
    x[7, 9] = np.inf
    x[8, 11] = np.nan
    dw, _ = gpu_lib.linear_backward_weight(dev(dy, "bf16"), dev(x, "bf16"), x_act=act)
    got = host(dw)
    assert np.array_equal(got[:, 9], np.sign(dy[7]) * np.inf)
    assert np.isnan(got[:, 11]).all()
    keep = [j for j in range(56) if j not in (9, 11)]
    assert np.isfinite(got[:, keep]).all()


def test_bf16_result_repeats_the_rounded_operand(gpu_lib):
    """A bf16 result takes the activation rounded once, as a bf16 forward product
    read it: bit for bit the gradient of the tensor that the forward pass made."""
    import torch
    log("recomputed activation, bf16 result")
    r = np.random.default_rng(6)
    dy, x = dev(r.standard_normal((150, 72)), "bf16"), dev(r.standard_normal((150, 88)), "bf16")
    q = gpu_lib.q8_quantize(x, "e4m3")
    a = gpu_lib.q8_dequantize(q, act="silu")
    got, _ = gpu_lib.linear_backward_weight(dy, q, x_act="silu", dtype=torch.bfloat16)
    want, _ = gpu_lib.linear_backward_weight(dy, a, dtype=torch.bfloat16)
    assert torch.equal(got, want)
