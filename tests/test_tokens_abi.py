"""Refusals of the token calls (host only), and their float64 oracle pinned.

Invalid calls use fake, never-dereferenced device addresses, as in test_abi.
"""
import ctypes

import numpy as np
import pytest

import matrix_aware_optimizers_amd as mao
from oracle import tokens as ref
from tests.test_abi import (E_ALIAS, E_DTYPE, E_HPARAM, E_LAYOUT, E_NULL, E_SHAPE, FAKE,
                            needs_no_gpu)

MB = 1 << 20


def m(i, rows, cols, ld=None, dtype=mao.F32, off=0):
    return mao.Mat(FAKE + i * MB + off, rows, cols, ld or (cols + 7) // 8 * 8, dtype)


def p(i, off=0):
    return ctypes.c_void_p(FAKE + i * MB + off)


@needs_no_gpu
def test_forward_refusals():
    lib = mao.load()

    def fwd(X=m(0, 4, 40), t=p(1), lp=p(2), ent=p(3), st=p(4), top=5, tl=p(5), ti=p(6)):
        return lib.mao_token_logprobs(X, t, lp, ent, st, top, tl, ti, None)

    assert fwd(X=m(0, 0, 40)) == E_SHAPE
    assert fwd(X=m(0, 4, 40, dtype=2)) == E_DTYPE
    assert fwd(X=m(0, 4, 40, ld=44)) == E_LAYOUT
    assert fwd(X=m(0, 4, 40, off=8)) == E_LAYOUT
    assert fwd(t=None) == E_NULL
    assert fwd(lp=None) == E_NULL
    assert fwd(top=0) == E_NULL  # alternatives' results without alternatives
    assert fwd(tl=None) == E_NULL
    assert fwd(ti=None) == E_NULL
    assert fwd(t=None, lp=None, ent=None, st=None, top=0, tl=None, ti=None) == E_NULL
    assert fwd(top=33) == E_HPARAM
    assert fwd(top=-1) == E_HPARAM
    assert fwd(X=m(0, 4, 3), top=4) == E_HPARAM
    assert fwd(t=p(1, 4)) == E_LAYOUT
    assert fwd(st=p(4, 2)) == E_LAYOUT
    assert fwd(ti=p(6, 4)) == E_LAYOUT
    assert fwd(lp=p(0, 16)) == E_ALIAS
    assert fwd(ent=p(4, 28)) == E_ALIAS  # the last of 8 statistics
    assert fwd(ti=p(1)) == E_ALIAS


@needs_no_gpu
def test_backward_refusals():
    lib = mao.load()

    def bwd(X=m(0, 4, 40), t=p(1), st=p(2), ent=p(3), dlp=p(4), de=p(5), dl=p(6), dX=m(7, 4, 40)):
        return lib.mao_token_logprobs_backward(X, t, st, ent, dlp, de, dl, dX, None)

    assert bwd(dX=m(7, 4, 41)) == E_SHAPE
    assert bwd(st=None) == E_NULL
    assert bwd(ent=None) == E_NULL
    assert bwd(t=None) == E_NULL
    assert bwd(dlp=None, de=None, dl=None) == E_NULL
    assert bwd(dl=p(6, 1)) == E_LAYOUT
    assert bwd(dX=m(0, 4, 40, off=16)) == E_ALIAS
    assert bwd(dX=m(0, 4, 40, dtype=mao.BF16)) == E_ALIAS  # in place needs one type
    assert bwd(dX=m(2, 4, 40)) == E_ALIAS

    def loss(X=m(0, 4, 40), t=p(1), w=p(2), lp=p(3), dX=m(4, 4, 40)):
        return lib.mao_token_loss(X, t, w, lp, dX, None)

    assert loss(t=None) == E_NULL
    assert loss(dX=m(4, 5, 40)) == E_SHAPE
    assert loss(w=p(2, 2)) == E_LAYOUT
    assert loss(t=p(1, 4)) == E_LAYOUT
    assert loss(dX=m(0, 4, 40, ld=48)) == E_ALIAS
    assert loss(lp=p(4, 4)) == E_ALIAS
    assert loss(lp=p(2)) == E_ALIAS


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 32))
    with pytest.raises(ValueError):
        mao.token_logprobs(x)
    with pytest.raises(ValueError):
        mao.token_loss(x, None)


def test_oracle_closed_forms():
    lp, ent, big, log_s, _ = ref.forward(np.full((1, 8), 3.0), [5])
    assert np.allclose([lp[0], ent[0], big[0], log_s[0]], [-np.log(8), np.log(8), 3.0, np.log(8)])
    x = np.full((1, 8), -np.inf)
    x[0, 2] = 1.0
    lp, ent, _, _, _ = ref.forward(x, [2])
    assert lp[0] == 0 and ent[0] == 0
    assert ref.top(np.array([[1.0, 3.0, 3.0, 2.0, 3.0]]), 4).tolist() == [[1, 2, 4, 3]]


def test_oracle_gradient_by_differences():
    r = np.random.default_rng(2)
    x = r.standard_normal((3, 11)) * 2
    x[1, 4] = -np.inf
    t = np.array([3, 0, -1])
    a, b, c = r.standard_normal((3, 3))

    def value(z):
        lp, ent, big, log_s, _ = ref.forward(z, t)
        return (a * lp + b * ent + c * (big + log_s)).sum()

    g = ref.backward(x, t, a, b, c)
    assert g[1, 4] == 0
    for i in range(3):
        for j in range(11):
            if np.isinf(x[i, j]):
                continue
            h = 1e-5
            up, down = x.copy(), x.copy()
            up[i, j] += h
            down[i, j] -= h
            assert abs((value(up) - value(down)) / (2 * h) - g[i, j]) < 1e-8
