"""Layer operators on inputs that take several rounds of the grid (GPU).

The norm and checkpoint kernels run a fixed number of workgroups at most, each over
several rows or pieces in turn, the next one loaded ahead. Here every size takes two
rounds or more (the norms' backward pass three or more), against float64 on the GPU.
Bounds as in test_gpu_layers: u = 2^-24, a row's sums with at most 84 roundings,
column sums with one per row.
"""
import pytest

from tests.helpers import log
from tests.test_gpu_layers import B, U

pytestmark = pytest.mark.gpu


def _input(seed, rows, cols, dtype, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda") * scale
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x += 0.5 * scale * torch.randn((rows, 1), generator=g, device="cuda")
    buf = torch.full((rows, (cols + 7) // 8 * 8), float("nan"), device="cuda",
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    buf[:, :cols] = x
    return buf[:, :cols]


def _check(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (what, int((err > bound).sum()), float((err / bound).max()))


def _rounded(want, bound, dtype):
    return bound + (B if dtype == "bf16" else U) * (want.abs() + bound) + 1e-37


def _norm(x, eps=1e-5):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    return mean, 1.0 / (d.square().mean(1) + eps).sqrt()


# threads per row 64 (one to four runs each), 256, 512, 1024
FORWARD = [(16390, 300), (16385, 1000), (16385, 1536), (8200, 2040), (4200, 4100), (2100, 8000),
           (1100, 16392), (1030, 30000)]
# threads per row 64, 128, 192, 256, 512, 1024 (one, two and four runs)
BACKWARD = [(12300, 400), (6200, 1000), (16385, 1536), (3100, 2000), (1600, 3000), (2100, 4100),
            (600, 8200), (600, 20001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", FORWARD)
def test_layer_norm_rounds(gpu_lib, rows, cols, dtype):
    import torch
    log(f"norm rounds {rows} x {cols} {dtype}")
    x = _input(rows, rows, cols, dtype)
    gamma = torch.linspace(0.5, 1.5, cols, device="cuda")
    beta = torch.linspace(-0.2, 0.3, cols, device="cuda")
    y, mean, rstd = gpu_lib.layer_norm(x, gamma, beta)
    wm, wr = _norm(x)
    xd = x.double()
    mag = xd.abs().mean(1) + wm.abs()
    em = 84 * U * mag
    _check(mean, wm, em, "mean")
    er = wr * (90 * U + em * wr * 1.01 + 4 * U * mag * wr)
    _check(rstd, wr, er, "rstd")
    wy = (xd - wm[:, None]) * wr[:, None] * gamma.double() + beta.double()
    xh = (xd - wm[:, None]).abs() * wr[:, None]
    by = gamma.double() * (((em + 2 * U * mag) * wr)[:, None] + xh * ((er / wr)[:, None] + 4 * U))
    _check(y, wy, _rounded(wy, by + 4 * U * beta.double().abs(), dtype), "y")


@pytest.mark.parametrize("dtype,saved", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "int8")])
@pytest.mark.parametrize("rows,cols", BACKWARD)
def test_layer_norm_backward_rounds(gpu_lib, rows, cols, dtype, saved):
    import torch
    log(f"norm backward rounds {rows} x {cols} {dtype} {saved}")
    x = _input(rows + 1, rows, cols, dtype)
    dy, add = (_input(rows + i, rows, cols, dtype, 1e-2) for i in (2, 3))
    gamma = torch.linspace(0.5, 1.5, cols, device="cuda")
    mean, rstd = (t.float() for t in _norm(x))
    kept = x
    xd = x.double()
    if saved == "int8":
        kept = gpu_lib.q8_quantize(x)
        xd = _values(kept)
    dx, dg, db = gpu_lib.layer_norm_backward(dy, kept, gamma, mean, rstd, add=add)
    m, s, d, a = mean.double()[:, None], rstd.double()[:, None], dy.double(), add.double()
    xh, g = (xd - m) * s, d * gamma.double()
    want = s * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) + a
    exh = U * (xd.abs() + m.abs()) * s + 3 * U * xh.abs()
    ga, xa = g.abs(), xh.abs()
    s0, s1 = ga.mean(1, keepdim=True), (ga * xa).mean(1, keepdim=True)
    e1 = 90 * U * s1 + (ga * exh).mean(1, keepdim=True)
    bound = s * (3 * U * ga + 90 * U * s0 + exh * s1 + xa * e1 + 4 * U * (ga + s0 + xa * s1))
    _check(dx, want, _rounded(want, bound + U * want.abs(), dtype), "dx")
    _check(dg, (d * xh).sum(0), (rows + 8) * U * (d * xh).abs().sum(0) + (d.abs() * exh).sum(0),
           "dgamma")
    _check(db, d.sum(0), (rows + 8) * U * d.abs().sum(0), "dbeta")


def _values(q):
    import torch
    s = torch.exp2(q.scales.double() - 127).repeat_interleave(32, 1)[:, :q.codes.shape[1]]
    return q.codes.to(torch.float32).double() * s


def _stored(x, fmt):
    """What a checkpoint of x stands for, in float64: per 32 columns the smallest power
    of two that keeps the rounded codes in range, each value at its nearest step, ties
    to even."""
    import torch
    rows, cols = x.shape
    nb = (cols + 31) // 32
    v = torch.zeros((rows, nb * 32), dtype=torch.float64, device="cuda")
    v[:, :cols] = x
    v = v.view(rows, nb, 32)
    top = v.abs().amax(2, keepdim=True)
    one = torch.ones_like(top)
    if fmt == "int8":
        step = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, one))) - 7)
        step = torch.where(torch.round(top / step) > 127, 2 * step, step)
        step = step.clamp(min=2.0 ** -126)
        w = torch.round(v / step) * step
    else:
        sc = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, one))) - 9)
        sc = torch.where(top / sc > 464, 2 * sc, sc).clamp(min=2.0 ** -124)
        a = v / sc
        e = torch.floor(torch.log2(torch.where(a == 0, torch.ones_like(a), a.abs()))).clamp(min=-6)
        w = torch.round(a / torch.exp2(e - 3)) * torch.exp2(e - 3) * sc
    return torch.where(top > 0, w, torch.zeros_like(w)).view(rows, nb * 32)[:, :cols]


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "f32")])
def test_checkpoint_rounds(gpu_lib, fmt, dtype):
    import torch
    log(f"checkpoint rounds {fmt} {dtype}")
    x = _input(5, 16391, 6151, dtype)
    q = gpu_lib.q8_quantize(x, fmt)
    want = _stored(x, fmt)
    assert torch.equal(_values(q), want)
    for t in (torch.bfloat16, torch.float32):
        assert torch.equal(gpu_lib.q8_dequantize(q, dtype=t).double(), want)
    z = gpu_lib.q8_dequantize(q, act="silu", dtype=torch.float32).double()
    _check(z, want * torch.sigmoid(want), 2e-6 * want.abs().clamp(min=1), "silu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu"])
def test_recomputed_activation_rounds(gpu_lib, act, dtype):
    """The activation of a saved tensor, rebuilt for the weight gradient. Row i of dY has
    one value, in column i mod 128, so a result adds 129 products at most and one wrong
    element of the rebuilt operand stands out of the bound."""
    import torch
    log(f"recomputed activation rounds {act} {dtype}")
    rows, cols, n = 16391, 6151, 128
    x = _input(6, rows, cols, dtype)
    i = torch.arange(rows, device="cuda")
    dy = torch.zeros((rows, n), device="cuda", dtype=x.dtype)
    dy[i, i % n] = 1 + (i % 5).to(x.dtype)
    dw, _ = gpu_lib.linear_backward_weight(dy, x, x_act=act, dbias=False)
    xd = x.double()
    a = xd.clamp(min=0) if act == "relu" else xd * torch.sigmoid(xd)
    want = torch.matmul(dy.double().t().contiguous(), a)
    mag = torch.matmul(dy.double().t().contiguous(), a.abs())
    bound = (129 + 12) * U * mag * (1 + B)
    if act != "relu":
        # the activation's own error, and (bf16) what its two parts leave of it
        e = 2e-6 * xd.abs().clamp(min=1) + (B * B if dtype == "bf16" else U) * a.abs()
        bound = bound + torch.matmul(dy.double().t().contiguous(), e)
    _check(dw, want, bound + 1e-37, "dw")
