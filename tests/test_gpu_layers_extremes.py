"""Activations far out, and rows with infinities and NaN (GPU).

A one-column identity layer shows an activation alone: x (n x 1) times a weight of one
is exact in fp32, so linear gives act(x), and the input gradient of ones gives act'(x).
r = 2^-24 is the rounding of one fp32 operation.
"""
import numpy as np
import pytest

from oracle import layers as ref
from tests.helpers import log
from tests.test_gpu_layers import ACTS, dev, host, vec

pytestmark = pytest.mark.gpu

R = 2.0 ** -24


def _value(lib, x, act):
    import torch
    one = dev(np.ones((1, 1)), "f32")
    return host(lib.linear(dev(x[:, None], "f32"), one, act=act))[:, 0]


def _slope(lib, x, act):
    one = dev(np.ones((1, 1)), "f32")
    return host(lib.linear_backward_input(dev(np.ones((len(x), 1)), "f32"), one, act=act,
                                          preact=dev(x[:, None], "f32")))[:, 0]


# a: the tail's exponent. Its constants, the steps that make it and the product that
# takes it to base 2 each round once: 2, 7 and 6 (twice 3, a square) times r, relative.
# exp2 and the reciprocal are off by 2 r each, the other operations by r.
TAILS = {"silu": (lambda z: np.abs(z), 2, 0.0, 80.0),
         "gelu_tanh": (lambda z: np.abs(2 * ref.GELU_C * (z + 0.044715 * z ** 3)), 7, 0.0, 9.0),
         "gelu": (lambda z: z * z / 2, 6, 4e-7, 12.5)}


@pytest.mark.parametrize("rows", [16, 20000])
@pytest.mark.parametrize("act", sorted(TAILS))
def test_negative_tails_keep_relative_accuracy(gpu_lib, act, rows):
    """... by the token kernel and by the tiles"""
    log(f"tail {act} {rows}")
    exponent, per_a, fit, far = TAILS[act]
    x = -np.linspace(0.01, far, rows).astype(np.float32)
    want = ref.act(x, act)
    bound = (fit + (per_a * exponent(x.astype(np.float64)) + 8) * R) * np.abs(want)
    got = _value(gpu_lib, x, act)
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


FAR = np.array([7.9, 8.1, 12.0, 19.9, 29.9, 30.0, 30.1, 31.0, 60.0, 87.0, 89.0, 119.0, 120.0, 121.0,
                1e3, 1e6, 1e18, 1e25, 3e38], np.float32)


@pytest.mark.parametrize("act", ACTS[1:])
def test_values_and_slopes_far_out(gpu_lib, act):
    """On both sides of every clamp."""
    log(f"far out {act}")
    x = np.concatenate([FAR, -FAR])
    x64 = np.clip(x.astype(np.float64), -1e90, 1e90)
    want = ref.act(x64, act) if act != "gelu_tanh" else np.where(x > 100, x64, np.where(
        x < -100, 0.0, ref.act(np.clip(x64, -100, 100), act)))
    got = _value(gpu_lib, x, act)
    assert (np.abs(got - want) <= 2e-6 * np.maximum(1, np.abs(x64))).all()
    slope = ref.act_slope(np.clip(x64, -200, 200), act)
    got = _slope(gpu_lib, x, act)
    assert (np.abs(got - slope) <= 2e-6 * np.minimum(np.maximum(1, np.abs(x64)), 200)).all()


@pytest.mark.parametrize("act", ACTS[1:])
def test_infinities_and_nan_through_activations(gpu_lib, act):
    """+inf stays; the smooth ones' z times 0 is NaN at -inf (as the formula is), relu's 0
    there; slopes are the limits; NaN stays NaN in both."""
    log(f"inf and nan {act}")
    x = np.array([np.inf, -np.inf, np.nan, 1.0], np.float32)
    y, s = _value(gpu_lib, x, act), _slope(gpu_lib, x, act)
    assert y[0] == np.inf and np.isnan(y[2]) and np.isfinite(y[3])
    assert y[1] == 0 if act == "relu" else np.isnan(y[1])
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and np.isfinite(s[3])


@pytest.mark.parametrize("shape", [(9, 72), (7, 1000), (6, 3001), (5, 9000)])
def test_norm_rows_with_infinity_or_nan(gpu_lib, shape):
    """A row with one is NaN throughout; the rows beside it are untouched."""
    import torch
    log(f"norm inf and nan {shape}")
    r = np.random.default_rng(1)
    x = r.standard_normal(shape).astype(np.float32)
    dy = r.standard_normal(shape).astype(np.float32)
    gamma = vec(r.standard_normal(shape[1]))
    clean, mean, rstd = gpu_lib.layer_norm(dev(x, "f32"), gamma, None)
    cdx, _, _ = gpu_lib.layer_norm_backward(dev(dy, "f32"), dev(x, "f32"), gamma, mean, rstd)
    bad = x.copy()
    bad[1, 3], bad[3, -1] = np.inf, np.nan
    y, m, s = gpu_lib.layer_norm(dev(bad, "f32"), gamma, None)
    dx, dg, _ = gpu_lib.layer_norm_backward(dev(dy, "f32"), dev(bad, "f32"), gamma, m, s)
    for i in range(shape[0]):
        if i in (1, 3):
            assert torch.isnan(y[i]).all() and torch.isnan(s[i]) and torch.isnan(dx[i]).all()
        else:
            assert torch.equal(y[i], clean[i]) and torch.equal(dx[i], cdx[i])
            assert m[i] == mean[i] and s[i] == rstd[i]
    assert torch.isnan(dg).all()


def test_two_host_threads(gpu_lib):
    """Two threads, each on a stream of its own, and both on one stream."""
    import threading

    import torch
    from tests.test_gpu_layers import _mlp_calls, _mlp_data
    log("two host threads")
    data = [_mlp_data(333, 264, 1000), _mlp_data(70, 136, 520)]
    want = [_mlp_calls(gpu_lib, t) for t in data]
    torch.cuda.synchronize()
    own = [torch.cuda.Stream(), torch.cuda.Stream()]
    for streams in (own, [own[0], own[0]]):
        got, failed = [[], []], []

        def work(i):
            try:
                with torch.cuda.stream(streams[i]):
                    for _ in range(20):
                        got[i].append(_mlp_calls(gpu_lib, data[i]))
            except BaseException as e:  # noqa: BLE001 (shown below)
                failed.append(e)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        for i in range(2):
            for outs in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
