"""The linear layer's products on every tile shape and with K split (GPU).

Ragged sizes for which the cut by estimated time comes out (or came out, with earlier
constants of the estimate) as each tile shape, alone or with K split over workgroups; each product against float64 (torch, on the GPU)
with the bounds of test_gpu_layers: (K + 8) 2^-24 of the magnitudes multiplied, then
one rounding of the result.
"""
import math

import pytest

from tests.helpers import log
from tests.test_gpu_layers import U

pytestmark = pytest.mark.gpu


def _rows(t):
    import torch
    r, c = t.shape
    buf = torch.full((r, (c + 7) // 8 * 8), math.nan, dtype=t.dtype, device="cuda")
    buf[:, :c] = t
    return buf[:, :c]


def _normal(g, r, c, scale=1.0, dtype="bf16"):
    import torch
    x = torch.randn((r, c), generator=g, device="cuda") * scale
    return _rows(x.bfloat16() if dtype == "bf16" else x)


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _check(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


def _gelu_tanh(z):
    import torch
    s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    ds = s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return z * s, s + z * ds


# 128x128, 128x128 split, 128x192, split, 192x128, split, 256x192, 256x256, split
FWD = [(123, 77, 88), (104, 790, 68), (674, 344, 5453), (5621, 3205, 141), (938, 327, 4325),
       (140, 3469, 5612), (3896, 79, 2079), (6184, 71, 2000), (5008, 5977, 1179),
       (1545, 69, 2634), (605, 4136, 775), (1009, 514, 5383), (412, 4024, 2760), (2227, 133, 2223),
       (133, 5185, 2774), (455, 5113, 4167), (67, 1896, 87)]
FWD += [(585, 65, 4933), (616, 3431, 838), (2899, 130, 4147), (430, 3523, 2697), (644, 565, 5400),
        (653, 3235, 1798), (391, 5645, 3255), (645, 5125, 5581)]
FWD += [(4383, 102, 5508), (517, 5000, 5158), (4448, 4777, 581)]
FWD32 = [(1545, 69, 2634), (3685, 1335, 1129), (123, 77, 88), (77, 468, 143)]
FWD32 += [(8410, 845, 462), (91, 343, 98)]


@pytest.mark.parametrize("rows,k,n,dtype", [(*s, "bf16") for s in FWD] + [(*s, "f32") for s in FWD32])
def test_forward_tiles(gpu_lib, rows, k, n, dtype):
    import torch
    log(f"forward tiles {rows} {k} {n} {dtype}")
    B = U if dtype == "f32" else 2.0 ** -8
    g = _gen(rows)
    x, w = _normal(g, rows, k, 1, dtype), _normal(g, n, k, 1 / math.sqrt(k), dtype)
    bias, res = torch.randn(n, generator=g, device="cuda"), _normal(g, rows, n, 1, dtype)
    z = _normal(g, rows, n, 1, dtype)
    y = gpu_lib.linear(x, w, bias, act="gelu_tanh", residual=res, preact=z)
    xd, wt = x.double(), w.double().t().contiguous()
    wz = torch.matmul(xd, wt) + bias.double()
    bz = (k + 8) * U * torch.matmul(xd.abs(), wt.abs()) + 2 * U * (wz.abs() + bias.abs())
    _check(z, wz, bz + B * (wz.abs() + bz), "z")
    wy = _gelu_tanh(wz)[0] + res.double()
    by = 1.2 * bz + 2e-6 * wz.abs().clamp(min=1) + U * (wy.abs() + res.double().abs())
    _check(y, wy, by + B * (wy.abs() + by), "y")


DX = [(123, 77, 88), (142, 82, 883), (2219, 1994, 325), (910, 1305, 4768), (4987, 837, 324),
      (146, 5530, 3508), (6137, 1296, 71), (5567, 2188, 70), (4907, 1154, 5826),
      (5010, 709, 66), (591, 774, 4132), (6240, 950, 563), (386, 2730, 4050), (1289, 3416, 134),
      (131, 2815, 5189), (454, 4171, 5030), (2148, 5484, 72), (96, 76, 1655)]
DX += [(680, 4439, 70), (1377, 332, 3406), (404, 2699, 3289), (1038, 3718, 537), (660, 1868, 3233),
    (385, 3369, 5645), (659, 5454, 5553), (65, 98, 1493)]
DX += [(2907, 4048, 265), (3441, 1738, 5956), (3687, 652, 5065)]
DX32 = [(2474, 1800, 82), (723, 5954, 1337), (123, 77, 88), (69, 85, 424)]
DX32 += [(964, 4217, 946), (66, 104, 313)]


@pytest.mark.parametrize("rows,k,n,dtype", [(*s, "bf16") for s in DX] + [(*s, "f32") for s in DX32])
def test_input_gradient_tiles(gpu_lib, rows, k, n, dtype):
    import torch
    log(f"input gradient tiles {rows} {k} {n} {dtype}")
    B = U if dtype == "f32" else 2.0 ** -8
    g = _gen(rows + 1)
    dy, w = _normal(g, rows, n, 1, dtype), _normal(g, n, k, 1 / math.sqrt(n), dtype)
    add, z = _normal(g, rows, k, 1, dtype), _normal(g, rows, k, 2.0)
    z8 = gpu_lib.q8_quantize(z, "int8")
    dx = gpu_lib.linear_backward_input(dy, w, act="gelu_tanh", preact=z8, add=add)
    zv = z8.codes.double() * torch.exp2(z8.scales.double() - 127).repeat_interleave(32, 1)[:, :k]
    dd, wd = dy.double(), w.double().contiguous()
    p = torch.matmul(dd, wd)
    want = p * _gelu_tanh(zv)[1] + add.double()
    bound = 1.2 * (n + 8) * U * torch.matmul(dd.abs(), wd.abs()) + U * (want.abs() + add.double().abs())
    bound = bound + 2e-6 * zv.abs().clamp(min=1) * p.abs()
    _check(dx, want, bound + B * (want.abs() + bound), "dx")


DW = [(123, 77, 88), (1254, 90, 67), (338, 4623, 780), (4485, 1324, 908), (336, 775, 4922),
      (7193, 3460, 133), (67, 2321, 5181), (6640, 1160, 4962),
      (130, 2187, 1357), (6969, 322, 770), (450, 2460, 2316), (8439, 134, 2318), (129, 4587, 937),
      (3572, 1234, 1041), (67, 5065, 1559), (5736, 1723, 1233), (8257, 2391, 1176), (1612, 104, 81)]
DW += [(68, 1218, 2462), (4012, 1784, 195), (65, 5676, 2138), (3318, 2720, 389), (461, 3096, 1289),
    (3363, 1166, 1060), (4106, 546, 3658), (6338, 2372, 1200)]
DW += [(6086, 4453, 618), (376, 2150, 5641), (6930, 4925, 530)]
DW32 = [(65, 1389, 2993), (1422, 975, 4199), (123, 77, 88), (428, 81, 85)]
DW32 += [(939, 902, 4419)]


@pytest.mark.parametrize("rows,k,n,dtype", [(*s, "bf16") for s in DW] + [(*s, "f32") for s in DW32])
def test_weight_gradient_tiles(gpu_lib, rows, k, n, dtype):
    import torch
    log(f"weight gradient tiles {rows} {k} {n} {dtype}")
    g = _gen(rows + 2)
    dy, x = _normal(g, rows, n, 1, dtype), _normal(g, rows, k, 1, dtype)
    for out in (torch.float32, torch.bfloat16):
        dw, db = gpu_lib.linear_backward_weight(dy, x, dtype=out)
        dt, xd = dy.double().t().contiguous(), x.double().contiguous()
        want = torch.matmul(dt, xd)
        bound = (rows + 8) * U * torch.matmul(dt.abs(), xd.abs())
        r = 2.0 ** -8 if out == torch.bfloat16 else U
        _check(dw, want, bound + r * (want.abs() + bound), "dw")
        _check(db, dt.sum(1), (rows + 8) * U * dt.abs().sum(1), "dbias")
