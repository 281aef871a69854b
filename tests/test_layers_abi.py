"""Refusals of the layer operators' C entry points (host only), and the float64
forms they are tested against, pinned by differences.

Invalid calls use fake, never-dereferenced device addresses, as in test_abi; they
are skipped when a GPU is present.
"""
import ctypes
import math

import numpy as np
import pytest

import matrix_aware_optimizers_amd as mao
from oracle import layers as ref
from tests.test_abi import (E_ALIAS, E_DTYPE, E_HPARAM, E_LAYOUT, E_NULL, E_SHAPE, E_UNSUPPORTED,
                            E_WORKSPACE, FAKE, needs_no_gpu)

MB = 1 << 20


def m(i, rows, cols, ld=None, dtype=mao.F32, off=0):
    return mao.Mat(FAKE + i * MB + off, rows, cols, ld or (cols + 7) // 8 * 8, dtype)


def q(i, rows, cols, ld=None, lds=None, fmt=0, off=0):
    base = FAKE + i * MB
    return mao.Q8C(base + off, base + MB // 2, rows, cols, ld or (cols + 31) // 32 * 32,
                   lds or (cols + 31) // 32, fmt)


def p(i, off=0):
    return ctypes.c_void_p(FAKE + i * MB + off)


def by(x):
    return None if x is None else ctypes.byref(x)


@needs_no_gpu
def test_q8_refusals():
    lib = mao.load()

    def quant(X=m(0, 4, 40), X8=q(1, 4, 40)):
        return lib.mao_q8_quantize(X, by(X8), None)

    assert quant(X=mao.Mat(None, 4, 40, 40, 0)) == E_NULL
    assert quant(X8=None) == E_NULL
    assert quant(X=m(0, 0, 40)) == E_SHAPE
    assert quant(X8=q(1, 4, 41)) == E_SHAPE
    assert quant(X8=q(1, 4, 40, ld=40)) == E_LAYOUT
    assert quant(X8=q(1, 4, 40, lds=1)) == E_LAYOUT
    assert quant(X8=q(1, 4, 40, off=8)) == E_LAYOUT
    assert quant(X8=q(1, 4, 40, fmt=2)) == E_DTYPE
    assert quant(X=m(0, 4, 40, dtype=2)) == E_DTYPE
    assert quant(X8=q(0, 4, 40, off=64)) == E_ALIAS

    def deq(X8=q(1, 4, 40), act=0, Y=m(0, 4, 40)):
        return lib.mao_q8_dequantize(by(X8), act, Y, None)

    assert deq(act=5) == E_HPARAM
    assert deq(Y=m(0, 4, 39)) == E_SHAPE
    assert deq(Y=m(1, 4, 40)) == E_ALIAS


@needs_no_gpu
def test_layer_norm_refusals():
    lib = mao.load()

    def fwd(X=m(0, 4, 40), g=p(1), b=p(2), pd=0, eps=1e-5, Y=m(3, 4, 40), mean=p(4), rstd=p(5)):
        return lib.mao_layer_norm(X, g, b, pd, eps, Y, mean, rstd, None)

    assert fwd(Y=m(3, 4, 41)) == E_SHAPE
    assert fwd(eps=0.0) == E_HPARAM
    assert fwd(eps=float("inf")) == E_HPARAM
    assert fwd(pd=3) == E_DTYPE
    assert fwd(g=p(1, 4)) == E_LAYOUT
    assert fwd(mean=p(4, 2)) == E_LAYOUT
    assert fwd(Y=m(0, 4, 40)) == E_ALIAS
    assert fwd(mean=p(5)) == E_ALIAS
    wide = 32769
    assert fwd(X=m(0, 1, wide), Y=m(3, 1, wide)) == E_UNSUPPORTED

    need = lib.mao_layer_norm_backward_workspace_size(4, 40)
    assert need > 0 and lib.mao_layer_norm_backward_workspace_size(4, wide) == 0

    def bwd(dY=m(0, 4, 40), X=m(1, 4, 40), X8=None, g=p(2), mean=p(3), rstd=p(4), add=None,
            dX=m(5, 4, 40), dg=p(6), db=p(7), ws=p(8), n=need):
        return lib.mao_layer_norm_backward(dY, by(X), by(X8), g, 0, mean, rstd, by(add), dX, dg,
                                           db, ws, n, None)

    assert bwd(X=None) == E_NULL
    assert bwd(X8=q(9, 4, 40)) == E_NULL
    assert bwd(X=None, X8=q(9, 5, 40)) == E_SHAPE
    assert bwd(mean=None) == E_NULL
    assert bwd(add=m(9, 4, 32)) == E_SHAPE
    assert bwd(add=m(5, 4, 40, off=32)) == E_ALIAS
    assert bwd(dX=m(0, 4, 40)) == E_ALIAS
    assert bwd(dg=p(7)) == E_ALIAS
    assert bwd(ws=None) == E_WORKSPACE
    assert bwd(n=need - 1) == E_WORKSPACE
    assert bwd(ws=p(5)) == E_ALIAS


@needs_no_gpu
def test_linear_refusals():
    lib = mao.load()
    big = lib.mao_linear_workspace_size(100, 4000, 48, mao.BF16)
    assert big > 0  # few tiles, long K: split
    assert lib.mao_linear_workspace_size(5, 4000, 48, mao.BF16) == 0
    assert lib.mao_linear_workspace_size(100, 0, 48, mao.BF16) == 0
    assert lib.mao_linear_workspace_size(100, 8, 48, 9) == 0

    def fwd(X=m(0, 100, 40), W=m(1, 48, 40), bias=p(2), bd=0, act=1, res=None, Y=m(3, 100, 48),
            z=None, ws=p(6), n=big):
        return lib.mao_linear(X, W, bias, bd, act, by(res), Y, by(z), ws, n, None)

    assert fwd(W=m(1, 48, 39)) == E_SHAPE
    assert fwd(W=m(1, 48, 40, dtype=mao.BF16)) == E_DTYPE
    assert fwd(Y=m(3, 100, 47)) == E_SHAPE
    assert fwd(act=9) == E_HPARAM
    assert fwd(bias=p(2, 8)) == E_LAYOUT
    assert fwd(bd=4) == E_DTYPE
    assert fwd(res=m(4, 99, 48)) == E_SHAPE
    assert fwd(res=m(3, 100, 48, off=16)) == E_ALIAS
    assert fwd(z=m(3, 100, 48)) == E_ALIAS
    assert fwd(Y=m(0, 100, 48)) == E_ALIAS
    assert fwd(X=m(0, 100, 40, ld=44)) == E_LAYOUT
    X, W = m(0, 100, 4000, dtype=mao.BF16), m(1, 48, 4000, dtype=mao.BF16)
    assert fwd(X=X, W=W, ws=None) == E_WORKSPACE
    assert fwd(X=X, W=W, n=big - 1) == E_WORKSPACE
    assert fwd(X=X, W=W, ws=p(6, 16)) == E_WORKSPACE

    def dx(dY=m(0, 100, 48), W=m(1, 48, 40), act=1, Z=m(2, 100, 40), Z8=None, add=None,
           dX=m(3, 100, 40)):
        return lib.mao_linear_backward_input(dY, W, act, by(Z), by(Z8), by(add), dX, p(6), MB, None)

    assert dx(Z=None) == E_NULL
    assert dx(Z8=q(4, 100, 40)) == E_NULL
    assert dx(act=0) == E_NULL
    assert dx(Z=m(2, 100, 48)) == E_SHAPE
    assert dx(W=m(1, 40, 40)) == E_SHAPE
    assert dx(dX=m(2, 100, 40)) == E_ALIAS

    need = lib.mao_linear_backward_weight_workspace_size(100, 40, 48, mao.F32, 1)
    assert need > lib.mao_linear_backward_weight_workspace_size(100, 40, 48, mao.F32, 0) > 0

    def dw(dY=m(0, 100, 48), X=None, X8=q(1, 100, 40), act=0, dW=m(2, 48, 40), db=p(3), n=need):
        return lib.mao_linear_backward_weight(dY, by(X), by(X8), act, dW, db, 0, p(6), n, None)

    assert dw(X8=None) == E_NULL
    assert dw(X=m(4, 100, 40)) == E_NULL
    assert dw(X=m(4, 100, 40, dtype=mao.BF16), X8=None) == E_DTYPE
    assert dw(dW=m(2, 47, 40)) == E_SHAPE
    assert dw(act=-1) == E_HPARAM
    assert dw(n=need - 1) == E_WORKSPACE
    assert dw(db=p(2)) == E_ALIAS


@pytest.mark.parametrize("kind", ["relu", "gelu", "gelu_tanh", "silu"])
def test_oracle_slopes_are_the_activations_differences(kind):
    z = np.linspace(-9, 9, 1801) + 1e-3
    h = 1e-6
    d = (ref.act(z + h, kind) - ref.act(z - h, kind)) / (2 * h)
    assert np.abs(d - ref.act_slope(z, kind)).max() < 1e-8


def test_oracle_activations_against_their_printed_forms():
    z = np.linspace(-4, 4, 81)
    erf = np.array([math.erf(v / math.sqrt(2)) for v in z])
    assert np.allclose(ref.act(z, "gelu"), 0.5 * z * (1 + erf), atol=1e-14)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    assert np.allclose(ref.act(z, "gelu_tanh"), 0.5 * z * (1 + np.tanh(u)), atol=1e-14)
    assert np.allclose(ref.act(z, "silu"), z / (1 + np.exp(-z)), atol=1e-14)


def test_oracle_layer_norm_gradient_by_differences():
    r = np.random.default_rng(1)
    x, g, c = r.standard_normal((3, 10)), r.standard_normal(10), r.standard_normal((3, 10))
    _, mean, rstd = ref.layer_norm(x, g, 0.0, 1e-5)
    dx, dg, db = ref.layer_norm_backward(c, x, g, mean, rstd)
    h = 1e-6
    for i, j in ((0, 0), (1, 4), (2, 9)):
        e = np.zeros_like(x)
        e[i, j] = h
        d = (c * (ref.layer_norm(x + e, g, 0.0, 1e-5)[0]
                  - ref.layer_norm(x - e, g, 0.0, 1e-5)[0])).sum() / (2 * h)
        assert abs(d - dx[i, j]) < 1e-7
    assert np.allclose(db, c.sum(0)) and np.allclose(
        dg, (c * ref.layer_norm(x, 1.0, 0.0, 1e-5)[0]).sum(0))


def test_oracle_checkpoint_values():
    x = np.array([[127.0, -63.6, 0.5, 0.0] + [0.0] * 28, [128.0, 1.0, 0.9, -3.0] + [0.0] * 28])
    v = ref.q8_values(x, "int8")
    assert v[0, :4].tolist() == [127.0, -64.0, 0.0, 0.0]   # steps of 1, ties to even
    assert v[1, :4].tolist() == [128.0, 0.0, 0.0, -4.0]    # 127.5 < 128: steps of 2
    w = ref.q8_values(np.array([[448.0, 464.0 / 2, 17.0, 0.001]]), "e4m3")
    assert w[0].tolist() == [448.0, 224.0, 16.0, 0.001953125 * round(0.001 / 0.001953125)]
