"""Refusals of the join between two blocks (host only), and its float64 oracle pinned.

Invalid calls use fake, never-dereferenced device addresses, as in test_abi.
"""
import ctypes

import numpy as np
import pytest

import matrix_aware_optimizers_amd as mao
from oracle import residual as ref
from tests.test_abi import (E_ALIAS, E_DTYPE, E_HPARAM, E_LAYOUT, E_NULL, E_SHAPE, E_UNSUPPORTED,
                            E_WORKSPACE, FAKE, needs_no_gpu)

MB = 1 << 20
BF = mao.BF16


def m(i, rows=4, cols=40, ld=None, dtype=mao.F32, off=0):
    return mao.Mat(FAKE + i * MB + off, rows, cols, ld or (cols + 7) // 8 * 8, dtype)


def p(i, off=0):
    return ctypes.c_void_p(FAKE + i * MB + off)


def n(kind, gamma=None, beta=None, dtype=0, eps=1e-5):
    return mao.RowNormC(kind, gamma and gamma.value, beta and beta.value, dtype, eps)


def by(x):
    return None if x is None else ctypes.byref(x)


LAYER = n(1, p(10), p(11))
RMS = n(2, p(12))
NONE = n(0)


@needs_no_gpu
def test_forward_refusals():
    lib = mao.load()

    def fwd(X=m(0), B=m(1), post=LAYER, gate=p(2), gd=0, gates=None, xs=1.0, bs=1.0, pre=RMS, R=m(3),
            H=m(4), st=p(5)):
        return lib.mao_residual_norm(X, B, by(post), gate, gd, by(gates), xs, bs, by(pre), R, by(H),
                                     st, None)

    assert fwd(post=None) == E_NULL
    assert fwd(pre=None) == E_NULL
    assert fwd(H=None) == E_NULL
    assert fwd(pre=NONE) == E_NULL  # a result without its norm
    assert fwd(gates=m(6)) == E_NULL  # two gates
    assert fwd(B=mao.Mat(None, 4, 40, 40, 0)) == E_NULL
    assert fwd(X=m(0, 5)) == E_SHAPE
    assert fwd(R=m(3, 4, 41)) == E_SHAPE
    assert fwd(H=m(4, 3)) == E_SHAPE
    assert fwd(gate=None, gates=m(6, 4, 32)) == E_SHAPE
    assert fwd(R=m(3, dtype=BF)) == E_DTYPE  # R has X's type
    assert fwd(H=m(4, dtype=BF)) == E_DTYPE  # H has B's
    assert fwd(gate=None, gates=m(6, dtype=BF)) == E_DTYPE
    assert fwd(gd=2) == E_DTYPE
    assert fwd(post=n(1, p(10), p(11), 5)) == E_DTYPE
    assert fwd(post=n(3, p(10))) == E_HPARAM
    assert fwd(post=n(0, p(10))) == E_HPARAM  # parameters without a norm
    assert fwd(pre=n(2, p(12), p(13))) == E_HPARAM  # no offset in this kind
    assert fwd(pre=n(2, p(12), eps=0.0)) == E_HPARAM
    assert fwd(xs=float("nan")) == E_HPARAM
    assert fwd(bs=float("inf")) == E_HPARAM
    assert fwd(gate=p(2, 8)) == E_LAYOUT
    assert fwd(post=n(1, p(10, 4), p(11))) == E_LAYOUT
    assert fwd(st=p(5, 8)) == E_LAYOUT
    assert fwd(X=m(0, ld=44)) == E_LAYOUT
    assert fwd(R=m(1)) == E_ALIAS
    assert fwd(R=m(0, ld=48)) == E_ALIAS
    assert fwd(H=m(3)) == E_ALIAS
    assert fwd(H=m(10)) == E_ALIAS  # a parameter
    assert fwd(st=p(0)) == E_ALIAS
    wide = dict(X=m(0, 1, 16385), B=m(1, 1, 16385), R=m(3, 1, 16385), H=m(4, 1, 16385))
    assert fwd(**wide) == E_UNSUPPORTED


@needs_no_gpu
def test_backward_refusals():
    lib = mao.load()
    size = lib.mao_residual_norm_backward_workspace_size
    need = size(4, 40)
    assert need > 0 and size(0, 40) == size(4, 16385) == 0
    full = mao.ResidualNormSumsC(p(20).value, p(21).value, p(22).value, None, p(23).value)

    def bwd(dH=m(0), dR=m(1), B=m(2), R=m(3), st=p(4), post=LAYER, gate=p(5), gd=0, gates=None, xs=1.0,
            bs=1.0, pre=RMS, dX=m(6), dB=m(7), dG=None, sums=full, ws=p(8), size=need):
        return lib.mao_residual_norm_backward(by(dH), by(dR), B, by(R), st, by(post), gate, gd,
                                              by(gates), xs, bs, by(pre), dX, dB, by(dG), by(sums), ws,
                                              size, None)

    assert bwd(dH=None) == E_NULL
    assert bwd(R=None) == E_NULL
    assert bwd(st=None) == E_NULL
    assert bwd(dG=m(9)) == E_NULL  # no gates
    assert bwd(pre=NONE, dH=None, R=None, dR=None) == E_NULL
    assert bwd(pre=NONE) == E_NULL
    assert bwd(dB=m(7, 4, 41)) == E_SHAPE
    assert bwd(dR=m(1, 3)) == E_SHAPE
    assert bwd(dX=m(6, dtype=BF)) == E_DTYPE
    assert bwd(dH=m(0, dtype=BF)) == E_DTYPE
    assert bwd(dB=m(7, dtype=BF)) == E_DTYPE
    wrong = mao.ResidualNormSumsC
    assert bwd(sums=wrong(None, None, None, p(24).value, None)) == E_HPARAM  # rms has no offset
    assert bwd(post=NONE, sums=wrong(p(20).value, None, None, None, None)) == E_HPARAM
    assert bwd(gate=None, sums=wrong(None, None, None, None, p(20).value)) == E_HPARAM
    assert bwd(st=p(4, 4)) == E_LAYOUT
    assert bwd(sums=wrong(p(20, 2).value, None, None, None, None)) == E_LAYOUT
    assert bwd(ws=None) == E_WORKSPACE
    assert bwd(size=need - 1) == E_WORKSPACE
    assert bwd(dX=m(2)) == E_ALIAS
    assert bwd(dX=m(1, off=16)) == E_ALIAS  # dR itself or none of it
    assert bwd(dB=m(2)) == E_ALIAS
    assert bwd(sums=wrong(p(20).value, p(20).value, None, None, None)) == E_ALIAS
    assert bwd(ws=p(20)) == E_ALIAS
    assert bwd(gate=None, gates=m(9), dG=m(9), sums=None) == E_ALIAS


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 32))
    with pytest.raises(ValueError):
        mao.residual_norm(x, x)
    with pytest.raises(ValueError):
        mao.residual_norm(x, x, post="batch")
    with pytest.raises(ValueError):
        mao.residual_norm_backward(x, x, x, x, x, pre="group")


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
def test_oracle_gradient_by_differences(post, pre):
    r = np.random.default_rng(4)
    rows, cols, eps = 3, 7, 1e-3
    x, b, gate, wr, wh = r.standard_normal((5, rows, cols))
    g1, b1, g2, b2 = r.standard_normal((4, cols))
    xs, bs = 0.7, -1.3

    def kinds(q1, o1, q2, o2):
        return ((post, q1, o1 if post == "layer" else 0.0), (pre, q2, o2 if pre == "layer" else 0.0))

    def value(x, b, gate, q1, o1, q2, o2):
        n1, n2 = kinds(q1, o1, q2, o2)
        rr, hh, _ = ref.forward(x, b, gate, xs, bs, n1, n2, eps)
        return (wr * rr).sum() + ((wh * hh).sum() if pre != "none" else 0.0)

    args = [x, b, gate, g1, b1, g2, b2]
    n1, n2 = kinds(g1, b1, g2, b2)
    rr, hh, st = ref.forward(x, b, gate, xs, bs, n1, n2, eps)
    grads = ref.backward(wh, wr, b, rr, st, gate, xs, bs, n1, n2)
    for k, g in enumerate(grads):
        if g is None or (k == 4 and post != "layer") or (k == 6 and pre != "layer"):
            continue
        for i in np.ndindex(args[k].shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][i] += 1e-6
            down[k][i] -= 1e-6
            assert abs((value(*up) - value(*down)) / 2e-6 - g[i]) < 1e-6
