"""Every tile shape that the linear layer picks, alone and with K split, is among the
sizes of the GPU tests (host only).

The cut is an estimate with fitted constants: a change of them may move the sizes of
the tests to other tiles, which this shows.
"""
import ctypes
import math
import random

import pytest

import matrix_aware_optimizers_amd as mao
import tests.test_gpu_layers as layers
import tests.test_gpu_layers_dispatch as dispatch
import tests.test_gpu_layers_tiles as tiles
from tests.test_abi import E_DTYPE, E_HPARAM, E_NULL, E_SHAPE

FORWARD, INPUT, WEIGHT = 0, 1, 2
NAMES = ["forward", "input gradient", "weight gradient"]
# product, operand type, mixed
KINDS = [(p, t, x) for p in (FORWARD, INPUT, WEIGHT) for t in (mao.BF16, mao.F32) for x in (0, 1)
         if not (x and (p == WEIGHT or t == mao.F32))]


def cut(product, rows, k, n, dtype, mixed=0):
    r = [ctypes.c_int32() for _ in range(3)]
    s = mao.load().mao_dbg_linear_cut(product, rows, k, n, dtype, mixed, *map(ctypes.byref, r))
    assert s == 0
    return tuple(v.value for v in r)


def shape(*args):
    bm, bn, split = cut(*args)
    return bm, bn, split > 1


SETS = {(FORWARD, mao.BF16, 0): [tiles.FWD, layers.LINEAR_SHAPES,
                                 [(r, k, 133) for r, k, t in dispatch.TOKENS if t == "bf16"]],
        (FORWARD, mao.BF16, 1): [dispatch.MIXED, layers.LINEAR_SHAPES[:-2]],
        (FORWARD, mao.F32, 0): [tiles.FWD32, layers.LINEAR_SHAPES[:-2],
                                [(r, k, 133) for r, k, t in dispatch.TOKENS if t == "f32"]],
        (INPUT, mao.BF16, 0): [tiles.DX],
        (INPUT, mao.BF16, 1): [dispatch.MIXED_DX],
        (INPUT, mao.F32, 0): [tiles.DX32],
        (WEIGHT, mao.BF16, 0): [tiles.DW],
        (WEIGHT, mao.F32, 0): [tiles.DW32]}


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{NAMES[k[0]]}-{k[1]}-{k[2]}")
def test_tested_sizes_reach_what_drawn_sizes_reach(kind):
    product, dtype, mixed = kind
    rng = random.Random(kind[0] * 4 + kind[1] * 2 + kind[2])

    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    reached = {}
    for _ in range(30000):
        s = (size(1, 16384), size(1, 16384), size(1, 16384))
        reached.setdefault(shape(product, *s, dtype, mixed), s)
    tested = {shape(product, *s, dtype, mixed) for sizes in SETS[kind] for s in sizes}
    missing = {c: s for c, s in reached.items() if c not in tested}
    assert not missing, f"tile shapes (rows, columns, K split) and a size that takes each: {missing}"


def test_accumulated_weight_gradients_are_cut_both_ways():
    both = {shape(WEIGHT, *s, mao.BF16)[2] for s in dispatch.ADDED}
    assert both == {True, False}
    assert {shape(WEIGHT, *s, mao.F32)[2] for s in dispatch.ADDED} == {True, False}


def test_cut_and_workspace_agree():
    lib = mao.load()
    rng = random.Random(5)
    for _ in range(300):
        rows, k, n = (rng.randint(17, 5000) for _ in range(3))
        for dtype in (mao.BF16, mao.F32):
            need = 0
            for mixed in (0, 1):
                split = cut(FORWARD, rows, k, n, dtype, mixed)[2]
                need = max(need, split * rows * ((n + 7) // 8 * 8) * 4 if split > 1 else 0)
            assert lib.mao_linear_workspace_size(rows, k, n, dtype) == need


def test_refusals():
    lib = mao.load()
    r = [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
    assert lib.mao_dbg_linear_cut(3, 8, 8, 8, 0, 0, *r) == E_HPARAM
    assert lib.mao_dbg_linear_cut(0, 0, 8, 8, 0, 0, *r) == E_SHAPE
    assert lib.mao_dbg_linear_cut(0, 8, 8, 8, 7, 0, *r) == E_DTYPE
    assert lib.mao_dbg_linear_cut(0, 8, 8, 8, 0, 0, None, r[1], r[2]) == E_NULL
