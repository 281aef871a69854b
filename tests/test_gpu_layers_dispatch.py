"""Kernels that the linear layer picks by type and length, each run at least once (GPU).

Bounds as in test_gpu_layers_tiles: (K + 8) 2^-24 of the magnitudes multiplied, then one
rounding of the result. test_layers_cut checks on the host that these sizes and those
of test_gpu_layers_tiles reach every tile shape, alone and with K split.
"""
import math

import pytest

from tests.helpers import log
from tests.test_gpu_layers import U
from tests.test_gpu_layers_tiles import _check, _gelu_tanh, _gen, _normal

pytestmark = pytest.mark.gpu

# up to 16 rows: eight wavefronts from 4096 columns on in bf16 and 2048 in fp32, four
# below; ragged last steps
TOKENS = [(rows, k, dtype) for rows in (1, 3, 16)
          for k, dtype in ((4088, "bf16"), (4096, "bf16"), (4100, "bf16"), (6151, "bf16"),
                           (2040, "f32"), (2048, "f32"), (2051, "f32"), (5000, "f32"))]
# rows, k, n: bf16 products whose result, pre-activation and joining tensor are fp32
MIXED = [(2051, 771, 3077), (300, 100, 133), (90, 2000, 200), (1100, 5000, 1101), (700, 6000, 900)]
MIXED_DX = [(2051, 3077, 771), (300, 133, 100), (90, 200, 2000), (1100, 1101, 5000),
            (700, 900, 6000)]
# weight gradients that add to what is there: tiles alone, K split over the rows
ADDED = [(8439, 134, 2318), (130, 2187, 1357), (6930, 4925, 530), (5736, 1723, 1233), (40, 77, 88),
         (3000, 70, 90)]


@pytest.mark.parametrize("rows,k,dtype", TOKENS)
def test_tokens_over_long_rows(gpu_lib, rows, k, dtype):
    import torch
    log(f"tokens {rows} {k} {dtype}")
    n, r = 133, U if dtype == "f32" else 2.0 ** -8
    g = _gen(k + rows)
    x, w = _normal(g, rows, k, 1, dtype), _normal(g, n, k, 1 / math.sqrt(k), dtype)
    bias, res = torch.randn(n, generator=g, device="cuda"), _normal(g, rows, n, 1, dtype)
    z = _normal(g, rows, n, 1, dtype)
    y = gpu_lib.linear(x, w, bias, act="gelu_tanh", residual=res, preact=z)
    xd, wt = x.double(), w.double().t().contiguous()
    wz = torch.matmul(xd, wt) + bias.double()
    bz = (k + 8) * U * torch.matmul(xd.abs(), wt.abs()) + 2 * U * (wz.abs() + bias.abs())
    _check(z, wz, bz + r * (wz.abs() + bz), "z")
    wy = _gelu_tanh(wz)[0] + res.double()
    by = 1.2 * bz + 2e-6 * wz.abs().clamp(min=1) + U * (wy.abs() + res.double().abs())
    _check(y, wy, by + r * (wy.abs() + by), "y")


@pytest.mark.parametrize("rows,k,n", MIXED)
def test_bf16_forward_with_fp32_ends(gpu_lib, rows, k, n):
    import torch
    log(f"mixed forward {rows} {k} {n}")
    g = _gen(rows + k)
    x, w = _normal(g, rows, k), _normal(g, n, k, 1 / math.sqrt(k))
    bias, res = torch.randn(n, generator=g, device="cuda"), _normal(g, rows, n, 1, "f32")
    xd, wt = x.double(), w.double().t().contiguous()
    wz = torch.matmul(xd, wt) + bias.double()
    bz = (k + 8) * U * torch.matmul(xd.abs(), wt.abs()) + 2 * U * (wz.abs() + bias.abs())
    wy = _gelu_tanh(wz)[0] + res.double()
    by = 1.2 * bz + 2e-6 * wz.abs().clamp(min=1) + U * (wy.abs() + res.double().abs())
    for zt, ot in (("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")):
        z, out = _normal(g, rows, n, 1, zt), _normal(g, rows, n, 1, ot)
        y = gpu_lib.linear(x, w, bias, act="gelu_tanh", residual=res, preact=z, out=out)
        rz, ro = (U if t == "f32" else 2.0 ** -8 for t in (zt, ot))
        _check(z, wz, bz + rz * (wz.abs() + bz), "z")
        _check(y, wy, by + ro * (wy.abs() + by), "y")


@pytest.mark.parametrize("rows,k,n", MIXED_DX)
def test_bf16_input_gradient_with_fp32_ends(gpu_lib, rows, k, n):
    import torch
    log(f"mixed input gradient {rows} {k} {n}")
    g = _gen(rows + n)
    dy, w = _normal(g, rows, n), _normal(g, n, k, 1 / math.sqrt(n))
    add, z = _normal(g, rows, k, 1, "f32"), _normal(g, rows, k, 2.0, "f32")
    out = _normal(g, rows, k, 1, "f32")
    dx = gpu_lib.linear_backward_input(dy, w, act="gelu_tanh", preact=z, add=add, out=out)
    dd, wd, zd = dy.double(), w.double().contiguous(), z.double()
    p = torch.matmul(dd, wd)
    want = p * _gelu_tanh(zd)[1] + add.double()
    bound = 1.2 * (n + 8) * U * torch.matmul(dd.abs(), wd.abs()) + U * (want.abs() + add.double().abs())
    bound = bound + 2e-6 * zd.abs().clamp(min=1) * p.abs()
    _check(dx, want, bound + U * (want.abs() + bound), "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", ADDED)
def test_weight_gradient_adds_to_what_is_there(gpu_lib, rows, k, n, dtype):
    import torch
    log(f"accumulated weight gradient {rows} {k} {n} {dtype}")
    g = _gen(rows + 3)
    dy, x = _normal(g, rows, n, 1, dtype), _normal(g, rows, k, 1, dtype)
    dt, xd = dy.double().t().contiguous(), x.double().contiguous()
    p = torch.matmul(dt, xd)
    bp = (rows + 8) * U * torch.matmul(dt.abs(), xd.abs())
    for out in ("f32", "bf16"):
        first, firstb = _normal(g, n, k, 30, out), torch.randn(n, generator=g, device="cuda")
        dw, db = gpu_lib.padded(first.clone()), firstb.clone()
        gpu_lib.linear_backward_weight(dy, x, out=dw, dbias=db, accumulate=True)
        want = p + first.double()
        bound = bp + U * first.double().abs()
        r = 2.0 ** -8 if out == "bf16" else U
        _check(dw, want, bound + r * (want.abs() + bound), "dw")
        wb = dt.sum(1) + firstb.double()
        _check(db, wb, (rows + 8) * U * (dt.abs().sum(1) + firstb.double().abs()), "dbias")
