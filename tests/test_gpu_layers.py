"""Layer norm, the linear layer and 8-bit checkpoints against float64 (GPU).

Bounds follow from the arithmetic. u = 2^-24 is the rounding of one fp32
operation and B = 2^-8 the largest relative error of a value rounded to bf16.
A sum of K fp32 products differs from the exact one by at most (K + 8) u times
the sum of their magnitudes, whatever its order; the activations and their
slopes are evaluated to 2e-6 of max(1, |z|) (exponentials of arguments up to 30,
relative error 30 u times a few) and change by at most 1.2 times a change of z
(slopes: 1.1). Inputs are rounded to their type before either side reads them.
Storage between the columns and the next multiple of 8 holds NaN.
"""
import math

import numpy as np
import pytest

from oracle import layers as ref
from synth import bf16_round
from tests.helpers import log

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _dt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _round(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return bf16_round(x) if dtype == "bf16" else x


def dev(x, dtype, extra=0):
    """x on the GPU in rows padded to a multiple of 8 (+ extra), the pad NaN."""
    import torch
    r, c = x.shape
    ld = (c + 7) // 8 * 8 + extra
    buf = torch.full((r, ld), math.nan, dtype=_dt(dtype), device="cuda")
    buf[:, :c] = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to("cuda")
    return buf[:, :c]


def vec(x, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to("cuda").to(_dt(dtype))


def host(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def values(q):
    """float64 values of a Q8 from its codes and scales."""
    import torch
    c = q.codes.to(torch.float32).double().cpu().numpy()
    s = q.scales.cpu().numpy().astype(np.float64)
    return c * np.exp2(np.repeat(s - 127.0, 32, axis=1)[:, :c.shape[1]])


def check(got, want, bound, what):
    err = np.abs(host(got) - want)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err / np.maximum(bound, 1e-300))))


def rounded(want, bound, dtype):
    """Bound after one rounding of the result to its type."""
    return bound + (B if dtype == "bf16" else U) * (np.abs(want) + bound) + 1e-37


# ---- 8-bit checkpoints -----------------------------------------------------

def _q8_input(rows, cols, dtype, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * np.exp(3 * r.standard_normal((rows, 1)))
    x[:, ::37] *= 50.0
    x = x.astype(np.float32)
    x.reshape(-1)[::11] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2] *= np.float32(2.0 ** -120)
    return _round(x, dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (3, 32), (5, 33), (4, 48), (7, 1000), (130, 257)])
def test_q8_values(gpu_lib, shape, dtype, fmt):
    import torch
    log(f"q8 {shape} {dtype} {fmt}")
    x = _q8_input(*shape, dtype, 3)
    q = gpu_lib.q8_quantize(dev(x, dtype), fmt)
    want = ref.q8_values(x, fmt)
    assert np.array_equal(values(q), want)
    # every stored value is exact in bf16, so both read-backs are too
    for t in (torch.bfloat16, torch.float32):
        assert np.array_equal(host(gpu_lib.q8_dequantize(q, dtype=t)), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_q8_range_edges(gpu_lib, fmt):
    log(f"q8 edges {fmt}")
    # largest magnitudes on both sides of every rounding threshold
    tops = [127.0, 127.25, 127.4999, 127.5, 127.75, 128.0, 248.0, 255.0, 256.0, 448.0, 463.9,
            464.0, 464.1, 480.0, 511.0, 512.0, 1.0, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149, 3.3e38]
    x = np.zeros((len(tops), 40), np.float32)
    for i, t in enumerate(tops):
        x[i, 3] = -t
        x[i, 4:32] = t * np.linspace(-1, 1, 28)
        x[i, 35] = t * 0.3
    q = gpu_lib.q8_quantize(dev(x, "f32"), fmt)
    assert np.array_equal(values(q), ref.q8_values(x, fmt))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_q8_shows_nan_and_infinity(gpu_lib, fmt):
    import torch
    log(f"q8 nan {fmt}")
    x = np.ones((3, 96), np.float32)
    x[0, 40], x[1, 0], x[2, 95] = np.nan, np.inf, -np.inf
    q = gpu_lib.q8_quantize(dev(x, "f32"), fmt)
    got = host(gpu_lib.q8_dequantize(q, dtype=torch.float32))
    want = ref.q8_values(x, fmt)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


@pytest.mark.parametrize("act", ACTS[1:])
def test_q8_read_through_activation(gpu_lib, act):
    import torch
    log(f"q8 act {act}")
    x = _q8_input(9, 203, "bf16", 5)
    q = gpu_lib.q8_quantize(dev(x, "bf16"), "int8")
    z = values(q)
    check(gpu_lib.q8_dequantize(q, act=act, dtype=torch.float32), ref.act(z, act),
          2e-6 * np.maximum(1.0, np.abs(z)) * 1.0, act)


def test_q8_leaves_the_pad_alone(gpu_lib):
    import torch
    log("q8 pad")
    codes = torch.full((5, 64), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((5, 4), 99, dtype=torch.uint8, device="cuda")
    gpu_lib.q8_quantize(dev(_q8_input(5, 41, "f32", 1), "f32"),
                        out=gpu_lib.Q8(codes[:, :41], scales))
    assert (codes[:, 41:] == 77).all() and (scales[:, 2:] == 99).all()


# ---- layer norm ------------------------------------------------------------

NORM_SHAPES = [(1, 1), (2, 7), (3, 8), (5, 130), (67, 512), (33, 513), (300, 1536), (9, 1537),
               (7, 2049), (600, 4096), (5, 4104), (3, 8200), (2, 14336), (2, 20001)]


def _norm_input(rows, cols, dtype, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * np.exp(0.5 * r.standard_normal((rows, 1)))
    x += r.standard_normal((rows, 1))
    x[:, ::19] *= 6.0
    if rows > 1:
        x[0] = 0.0          # a padding token
    if rows > 2:
        x[2] = 3.25         # a constant row
    return _round(x, dtype), r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm(gpu_lib, shape, dtype):
    log(f"layer norm {shape} {dtype}")
    x, r = _norm_input(*shape, dtype, 7)
    n = shape[1]
    gamma, beta = 1 + 0.3 * r.standard_normal(n), 0.2 * r.standard_normal(n)
    gamma, beta = _round(gamma, dtype), _round(beta, dtype)
    y, mean, rstd = gpu_lib.layer_norm(dev(x, dtype, 8), vec(gamma, dtype), vec(beta, dtype),
                                       eps=1e-5)
    wy, wm, wr = ref.layer_norm(x, gamma, beta, 1e-5)
    # a sum held by 64 threads or more, V runs of 8 each: at most 64 + 20 roundings
    mag = np.abs(x).mean(axis=1) + np.abs(wm)
    em = 84 * U * mag
    check(mean, wm, em + 1e-30, "mean")
    # deviations carry the mean's error; the square root halves the relative
    # error of the variance
    er = wr * (90 * U + em * wr * 1.01 + 4 * U * mag * wr)
    check(rstd, wr, er, "rstd")
    xh = np.abs(x - wm[:, None]) * wr[:, None]
    by = np.abs(gamma)[None, :] * (((em + 2 * U * mag) * wr)[:, None]
                                   + xh * ((er / wr)[:, None] + 4 * U)) + 4 * U * np.abs(beta)
    check(y, wy, rounded(wy, by, dtype), "y")


def test_layer_norm_far_from_zero(gpu_lib):
    # the variance comes from deviations: an offset of 1000 costs 1000 u, not 1000^2 u
    log("layer norm offset")
    r = np.random.default_rng(2)
    x = (1000 + r.standard_normal((4, 777))).astype(np.float32)
    y, _, _ = gpu_lib.layer_norm(dev(x, "f32"))
    wy, _, _ = ref.layer_norm(x, 1.0, 0.0, 1e-5)
    assert np.abs(host(y) - wy).max() < 90 * U * 1000 * 1.5 * 4


def test_layer_norm_without_parameters_and_mixed_types(gpu_lib):
    import torch
    log("layer norm mixed")
    x, _ = _norm_input(11, 300, "f32", 4)
    out = torch.empty((11, 304), dtype=torch.bfloat16, device="cuda")[:, :300]
    y, mean, rstd = gpu_lib.layer_norm(dev(x, "f32"), out=out, stats=False)
    assert mean is None and rstd is None
    wy, _, _ = ref.layer_norm(x, 1.0, 0.0, 1e-5)
    check(y, wy, rounded(wy, 1e-4 * np.ones_like(wy), "bf16"), "y")


def _norm_backward_bound(dy, x, gamma, mean, rstd, rows, n):
    """Roundings of the two row sums and of xh, carried through the formula."""
    xh = np.abs(x - mean[:, None]) * rstd[:, None]
    exh = U * (np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None] + 3 * U * xh
    g = np.abs(dy * gamma)
    s0 = g.mean(axis=1, keepdims=True)
    s1 = (g * xh).mean(axis=1, keepdims=True)
    e1 = 90 * U * s1 + (g * exh).mean(axis=1, keepdims=True)
    bdx = rstd[:, None] * (3 * U * g + 90 * U * s0 + exh * s1 + xh * e1
                           + 4 * U * (g + s0 + xh * s1))
    bdg = (rows + 8) * U * np.abs(dy * xh).sum(axis=0) + np.abs(dy * exh).sum(axis=0)
    bdb = (rows + 8) * U * np.abs(dy).sum(axis=0)
    return bdx, bdg + 1e-30, bdb + 1e-30


@pytest.mark.parametrize("dtype,saved", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "int8"),
                                         ("bf16", "e4m3"), ("f32", "int8"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_backward(gpu_lib, shape, dtype, saved):
    log(f"layer norm backward {shape} {dtype} {saved}")
    rows, n = shape
    x, r = _norm_input(rows, n, "f32" if saved == "f32" else "bf16", 11)
    gamma = _round(1 + 0.3 * r.standard_normal(n), "f32")
    dy = _round(1e-2 * r.standard_normal(shape), dtype)
    add = _round(1e-2 * r.standard_normal(shape), dtype) if n % 2 else None
    _, mean, rstd = ref.layer_norm(x, 1.0, 0.0, 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    if saved in ("int8", "e4m3"):
        kept = gpu_lib.q8_quantize(dev(x, "bf16"), saved)
        x = values(kept)
    else:
        kept = dev(x, saved)
    dx, dg, db = gpu_lib.layer_norm_backward(
        dev(dy, dtype), kept, vec(gamma), vec(mean), vec(rstd),
        add=None if add is None else dev(add, dtype, 16))
    mean, rstd = mean.astype(np.float64), rstd.astype(np.float64)
    wdx, wdg, wdb = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    bdx, bdg, bdb = _norm_backward_bound(dy.astype(np.float64), x, gamma, mean, rstd, rows, n)
    if add is not None:
        wdx = wdx + add
        bdx = bdx + U * np.abs(wdx)
    check(dx, wdx, rounded(wdx, bdx, dtype), "dx")
    check(dg, wdg, bdg, "dgamma")
    check(db, wdb, bdb, "dbeta")


def test_layer_norm_gradient_against_differences(gpu_lib):
    """Directional differences of the float64 norm, L = sum c y."""
    log("layer norm differences")
    r = np.random.default_rng(3)
    x = r.standard_normal((6, 45)).astype(np.float32)
    gamma = (1 + 0.3 * r.standard_normal(45)).astype(np.float32)
    c = r.standard_normal((6, 45)).astype(np.float32)
    _, mean, rstd = gpu_lib.layer_norm(dev(x, "f32"), vec(gamma), None)
    dx, dg, db = gpu_lib.layer_norm_backward(dev(c, "f32"), dev(x, "f32"), vec(gamma), mean, rstd)

    def loss(xx, gg, bb):
        return (c * ref.layer_norm(xx, gg, bb, 1e-5)[0]).sum()

    h = 1e-5
    for k in range(4):
        v, w, b = r.standard_normal((6, 45)), r.standard_normal(45), r.standard_normal(45)
        d = (loss(x + h * v, gamma + h * w, h * b) - loss(x - h * v, gamma - h * w, -h * b)) / (2 * h)
        got = (host(dx) * v).sum() + (host(dg) * w).sum() + (host(db) * b).sum()
        scale = np.abs(host(dx) * v).sum() + np.abs(host(dg) * w).sum() + np.abs(host(db) * b).sum()
        assert abs(d - got) < 1e-6 * scale


# ---- linear ----------------------------------------------------------------

# rows, k, n: single tokens, prompts, ragged tiles, a K below one slice, enough
# tiles for the large tile, a K split over workgroups
LINEAR_SHAPES = [(1, 1, 1), (1, 40, 17), (3, 1000, 130), (16, 264, 48), (17, 129, 33), (40, 600, 70),
                 (64, 1536, 96), (65, 70, 33), (130, 100, 257), (77, 2100, 200), (300, 520, 1000),
                 (3500, 200, 3601), (3601, 71, 3400)]


def _linear_data(rows, k, n, dtype, seed):
    r = np.random.default_rng(seed)
    x = _round(r.standard_normal((rows, k)), dtype)
    w = _round(r.standard_normal((n, k)) / math.sqrt(k), dtype)
    return x, w, r


def _product_bound(a, b, k):
    return (k + 8) * U * (np.abs(a).astype(np.float64) @ np.abs(b).astype(np.float64))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LINEAR_SHAPES[:-2])
def test_linear(gpu_lib, shape, dtype, act):
    import torch
    log(f"linear {shape} {dtype} {act}")
    rows, k, n = shape
    x, w, r = _linear_data(rows, k, n, dtype, 13)
    bias = _round(r.standard_normal(n), dtype)
    res = _round(r.standard_normal((rows, n)), dtype)
    z = dev(np.zeros((rows, n)), "f32", 8)
    y = gpu_lib.linear(dev(x, dtype, 16), dev(w, dtype, 8), vec(bias, dtype), act=act,
                       residual=dev(res, dtype, 8), preact=z)
    wy, wz = ref.linear(x, w, bias, act, res)
    bz = _product_bound(x, w.T, k) + 2 * U * (np.abs(wz) + np.abs(bias))
    check(z, wz, rounded(wz, bz, "f32"), "z")
    by = 1.2 * bz + (2e-6 * np.maximum(1, np.abs(wz)) if act not in ("none", "relu") else 0)
    by = by + U * (np.abs(wy) + np.abs(res))
    check(y, wy, rounded(wy, by, dtype), "y")
    # the residual may be the output
    io = dev(res, dtype, 8)
    again = gpu_lib.linear(dev(x, dtype, 16), dev(w, dtype, 8), vec(bias, dtype), act=act,
                           residual=io, out=io)
    assert torch.equal(again, y)


@pytest.mark.parametrize("shape", LINEAR_SHAPES[-2:])
def test_linear_large_tiles(gpu_lib, shape):
    log(f"linear large {shape}")
    rows, k, n = shape
    x, w, r = _linear_data(rows, k, n, "bf16", 17)
    bias = _round(r.standard_normal(n), "f32")
    y = gpu_lib.linear(dev(x, "bf16"), dev(w, "bf16"), vec(bias), act="gelu_tanh")
    wy, wz = ref.linear(x, w, bias, "gelu_tanh")
    bz = _product_bound(x, w.T, k) + 2 * U * (np.abs(wz) + np.abs(bias))
    check(y, wy, rounded(wy, 1.2 * bz + 2e-6 * np.maximum(1, np.abs(wz)), "bf16"), "y")


def test_linear_plain_and_mixed_outputs(gpu_lib):
    import torch
    log("linear mixed")
    x, w, _ = _linear_data(150, 88, 90, "bf16", 19)
    out = torch.empty((150, 96), dtype=torch.float32, device="cuda")[:, :90]
    y = gpu_lib.linear(dev(x, "bf16"), dev(w, "bf16"), out=out)
    wy, _ = ref.linear(x, w, 0.0)
    check(y, wy, rounded(wy, _product_bound(x, w.T, 88), "f32"), "y")


@pytest.mark.parametrize("rows", [5, 200])
def test_linear_keeps_nan_in_its_row(gpu_lib, rows):
    log(f"linear nan {rows}")
    x, w, _ = _linear_data(rows, 100, 60, "bf16", 23)
    x[3, 50] = np.nan
    x[4, 99] = np.inf
    y = host(gpu_lib.linear(dev(x, "bf16"), dev(w, "bf16")))
    assert np.isnan(y[3]).all() and not np.isfinite(y[4]).any()
    keep = [i for i in range(rows) if i not in (3, 4)]
    assert np.isfinite(y[keep]).all()


def _kept(gpu_lib, x, kind):
    """x as kept for the backward pass, and the values that stand there."""
    if kind in ("int8", "e4m3"):
        q = gpu_lib.q8_quantize(dev(x, "bf16"), kind)
        return q, values(q)
    x = _round(x, kind)
    return dev(x, kind), x.astype(np.float64)


@pytest.mark.parametrize("act,saved", [("none", None), ("relu", "bf16"), ("gelu", "int8"),
                                       ("gelu_tanh", "int8"), ("gelu_tanh", "f32"),
                                       ("silu", "e4m3")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LINEAR_SHAPES)
def test_linear_backward_input(gpu_lib, shape, dtype, act, saved):
    rows, k, n = shape
    if rows > 1000 and (dtype, act) not in (("bf16", "none"), ("bf16", "gelu_tanh")):
        pytest.skip("large tiles: two variants")
    log(f"linear backward input {shape} {dtype} {act} {saved}")
    r = np.random.default_rng(29)
    dy = _round(r.standard_normal((rows, n)), dtype)
    w = _round(r.standard_normal((n, k)) / math.sqrt(n), dtype)
    add = _round(r.standard_normal((rows, k)), dtype)
    kept, z = (None, 0.0)
    if saved:
        kept, z = _kept(gpu_lib, 2 * r.standard_normal((rows, k)), saved)
    dx = gpu_lib.linear_backward_input(dev(dy, dtype, 8), dev(w, dtype, 16), act=act, preact=kept,
                                       add=dev(add, dtype, 8))
    p = dy.astype(np.float64) @ w.astype(np.float64)
    want = p * ref.act_slope(z, act) + add
    bound = 1.2 * _product_bound(dy, w, n) + U * (np.abs(want) + np.abs(add))
    if act not in ("none", "relu"):
        bound = bound + 2e-6 * np.maximum(1, np.abs(z)) * np.abs(p)
    check(dx, want, rounded(want, bound, dtype), "dx")


@pytest.mark.parametrize("x_act,saved,out", [("none", "own", "f32"), ("none", "int8", "f32"),
                                             ("none", "e4m3", "bf16"), ("gelu_tanh", "int8", "bf16"),
                                             ("silu", "own", "f32")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LINEAR_SHAPES[:-2] + [(130, 3601, 3500), (71, 3400, 3601)])
def test_linear_backward_weight(gpu_lib, shape, dtype, x_act, saved, out):
    rows, k, n = shape
    if k > 3000 and (dtype, saved) != ("bf16", "own"):
        pytest.skip("large tiles: one variant")
    log(f"linear backward weight {shape} {dtype} {x_act} {saved} {out}")
    r = np.random.default_rng(31)
    dy = _round(r.standard_normal((rows, n)), dtype)
    kept, x = _kept(gpu_lib, r.standard_normal((rows, k)), dtype if saved == "own" else saved)
    dw, db = gpu_lib.linear_backward_weight(dev(dy, dtype, 8), kept, x_act=x_act, dtype=_dt(out))
    want, wb = ref.linear_backward_weight(dy, x, x_act)
    a = np.abs(ref.act(x, x_act))
    bound = _product_bound(dy.T, a, rows)
    if x_act != "none":
        # the rebuilt activation's own error, and its rounding to bf16
        ea = 2e-6 * np.maximum(1, np.abs(x)) + (B * a if dtype == "bf16" else U * a)
        bound = bound + np.abs(dy).T.astype(np.float64) @ ea
    check(dw, want, rounded(want, bound, out), "dw")
    check(db, wb, (rows + 8) * U * np.abs(dy).sum(axis=0) + 1e-30, "dbias")


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_backward_weight_accumulates(gpu_lib, out):
    log(f"accumulate {out}")
    r = np.random.default_rng(37)
    dy = [_round(r.standard_normal((90 + 40 * i, 70)), "bf16") for i in range(2)]
    x = [_round(r.standard_normal((90 + 40 * i, 133)), "bf16") for i in range(2)]
    dw, db = gpu_lib.linear_backward_weight(dev(dy[0], "bf16"), dev(x[0], "bf16"), dtype=_dt(out))
    first, firstb = host(dw), host(db)
    gpu_lib.linear_backward_weight(dev(dy[1], "bf16"), dev(x[1], "bf16"), out=dw, dbias=db,
                                   accumulate=True)
    p, pb = ref.linear_backward_weight(dy[1], x[1])
    want = first + p
    check(dw, want, rounded(want, _product_bound(dy[1].T, x[1], 130) + U * np.abs(first), out), "dw")
    check(db, firstb + pb, 140 * U * (np.abs(dy[1]).sum(axis=0) + np.abs(firstb)), "dbias")


def test_linear_gradients_against_differences(gpu_lib):
    """L = sum c act(x W1^T + b1) W2^T: directional differences in float64."""
    log("linear differences")
    r = np.random.default_rng(41)
    x, w1 = r.standard_normal((70, 20)), r.standard_normal((31, 20)) / 4
    w2, b1, c = r.standard_normal((12, 31)) / 5, r.standard_normal(31), r.standard_normal((70, 12))
    x, w1, w2, b1, c = [v.astype(np.float32) for v in (x, w1, w2, b1, c)]
    for act in ACTS[2:]:
        z = dev(np.zeros((70, 31)), "f32")
        a = gpu_lib.linear(dev(x, "f32"), dev(w1, "f32"), vec(b1), act=act, preact=z)
        dw2, _ = gpu_lib.linear_backward_weight(dev(c, "f32"), a)
        dz = gpu_lib.linear_backward_input(dev(c, "f32"), dev(w2, "f32"), act=act, preact=z)
        dw1, db1 = gpu_lib.linear_backward_weight(dz, dev(x, "f32"))
        dx = gpu_lib.linear_backward_input(dz, dev(w1, "f32"))
        grads = [host(g) for g in (dx, dw1, db1, dw2)]

        def loss(xx, ww, bb, w22):
            return (c * ref.linear(ref.linear(xx, ww, bb, act)[0], w22, 0.0)[0]).sum()

        h = 1e-5
        for _ in range(3):
            v = [r.standard_normal(g.shape) for g in grads]
            p = [x, w1, b1, w2]
            d = (loss(*[q + h * t for q, t in zip(p, v)])
                 - loss(*[q - h * t for q, t in zip(p, v)])) / (2 * h)
            got = sum((g * t).sum() for g, t in zip(grads, v))
            scale = sum(np.abs(g * t).sum() for g, t in zip(grads, v))
            assert abs(d - got) < 2e-6 * scale


# ---- streams, repeatability, graphs ----------------------------------------

def _mlp_calls(lib, t):
    h, mean, rstd = lib.layer_norm(t["x"], t["g"], t["b"])
    z = lib.empty_matrix(t["x"].shape[0], t["w1"].shape[0], t["x"].dtype, t["x"].device)
    a = lib.linear(h, t["w1"], t["b1"], act="gelu_tanh", preact=z)
    y = lib.linear(a, t["w2"], t["b2"], residual=t["x"])
    x8, h8, z8 = lib.q8_quantize(t["x"]), lib.q8_quantize(h), lib.q8_quantize(z)
    dw2, db2 = lib.linear_backward_weight(t["dy"], z8, x_act="gelu_tanh")
    dz = lib.linear_backward_input(t["dy"], t["w2"], act="gelu_tanh", preact=z8)
    dw1, db1 = lib.linear_backward_weight(dz, h8)
    dh = lib.linear_backward_input(dz, t["w1"])
    dx, dg, db = lib.layer_norm_backward(dh, x8, t["g"], mean, rstd, add=t["dy"])
    return [y, dx, dg, db, dw1, db1, dw2, db2]


def _mlp_data(rows, d, f):
    r = np.random.default_rng(43)
    n = r.standard_normal
    return {"x": dev(n((rows, d)), "bf16"), "dy": dev(n((rows, d)), "bf16"),
            "w1": dev(n((f, d)) / 10, "bf16"), "w2": dev(n((d, f)) / 20, "bf16"),
            "g": vec(1 + 0.1 * n(d)), "b": vec(0.1 * n(d)), "b1": vec(n(f)), "b2": vec(n(d))}


def test_layer_calls_repeat_bit_for_bit_on_any_stream(gpu_lib):
    import torch
    log("streams")
    t = _mlp_data(333, 264, 1000)
    first = _mlp_calls(gpu_lib, t)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(2):
        for s in (s1, s2):  # both streams at work at once, each with its workspace
            with torch.cuda.stream(s):
                outs.append(_mlp_calls(gpu_lib, t))
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(first, o):
            assert torch.equal(a, b)


def test_layer_calls_replay_in_a_graph(gpu_lib):
    import torch
    log("graph")
    t = _mlp_data(150, 136, 520)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _mlp_calls(gpu_lib, t)  # workspace of this stream
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = _mlp_calls(gpu_lib, t)
    for k in range(3):
        t["x"].copy_(t["x"] * 0.5 + k)
        g.replay()
        torch.cuda.synchronize()
        want = _mlp_calls(gpu_lib, t)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_binding_refuses_what_the_kernels_cannot_read(gpu_lib):
    import torch
    log("refusals")
    x = torch.zeros((4, 16), device="cuda")
    w = torch.zeros((8, 16), device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.linear(x.cpu(), w.cpu())
    with pytest.raises(ValueError):
        gpu_lib.linear(x, w.cpu())
    with pytest.raises(ValueError):
        gpu_lib.linear(x, w, torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.linear(x.t(), w)
    with pytest.raises(TypeError):
        gpu_lib.linear(x.half(), w.half())
    with pytest.raises(gpu_lib.MaoError):
        gpu_lib.linear(x, w.bfloat16())
    with pytest.raises(gpu_lib.MaoError):
        gpu_lib.linear(x, torch.zeros((8, 15), device="cuda"))
    with pytest.raises(gpu_lib.MaoError):
        gpu_lib.linear_backward_input(torch.zeros((4, 8), device="cuda"), w, act="gelu")
    with pytest.raises(gpu_lib.MaoError):
        gpu_lib.layer_norm(x, out=x)
    with pytest.raises(TypeError):
        gpu_lib.Q8(x, x)
    with pytest.raises(ValueError):
        gpu_lib.linear_backward_weight(x, x, accumulate=True)
