"""Refusals of the many-tensor AdamW step (host only), and the 8-bit states' oracle.

Invalid calls use fake, never-dereferenced device addresses, as in test_abi.
"""
import ctypes

import numpy as np
import pytest

import matrix_aware_optimizers_amd as mao
from oracle import adam8
from tests.test_abi import E_ALIAS, E_DTYPE, E_HPARAM, E_LAYOUT, E_NULL, E_SHAPE, FAKE, needs_no_gpu

MB = 1 << 20


def item(k=0, n=1000, state=0, wd=0, gd=0, lr=1e-3, decay=0.0, **at):
    a = {name: FAKE + (8 * k + j) * MB for j, name in enumerate(("w", "g", "m", "v", "ms", "vs"))}
    a.update(at)
    return mao.AdamwTensorC(a["w"], a["g"], a["m"], a["v"], a["ms"], a["vs"], n, wd, gd, state, lr,
                            decay)


def step(items, t=1, b1=0.9, b2=0.95, eps=1e-8, gs=None, count=None):
    arr = (mao.AdamwTensorC * max(1, len(items)))(*items) if items is not None else None
    return mao.load().adamw_step_many(len(items or []) if count is None else count, arr, t, b1, b2,
                                      eps, gs, None)


@needs_no_gpu
def test_step_refusals():
    assert step(None, count=1) == E_NULL
    assert step([]) == E_SHAPE
    assert step([item()], count=4097) == E_SHAPE
    assert step([item(n=-1)]) == E_SHAPE
    assert step([item(n=(1 << 40) + 1)]) == E_SHAPE
    for name in ("w", "g", "m", "v"):
        assert step([item(**{name: None})]) == E_NULL
        assert step([item(**{name: FAKE + 2})]) == E_LAYOUT  # fp32 at a half-word
    assert step([item(state=1, ms=None)]) == E_NULL
    assert step([item(state=1, vs=FAKE + 5 * MB + 1)]) == E_LAYOUT
    assert step([item(state=2)]) == E_DTYPE
    assert step([item(wd=2)]) == E_DTYPE
    assert step([item(gd=-1)]) == E_DTYPE
    assert step([item()], t=0) == E_HPARAM
    assert step([item()], b1=1.0) == E_HPARAM
    assert step([item()], b2=-0.1) == E_HPARAM
    assert step([item()], b2=float("nan")) == E_HPARAM
    assert step([item()], eps=0.0) == E_HPARAM
    assert step([item(lr=-1.0)]) == E_HPARAM
    assert step([item(decay=float("inf"))]) == E_HPARAM
    assert step([item()], gs=ctypes.c_void_p(FAKE + 50 * MB + 2)) == E_LAYOUT


@needs_no_gpu
def test_step_aliases():
    """No written buffer may share a byte with another; gradients may be shared."""
    assert step([item(0), item(1, w=FAKE + 999 * 4)]) == E_ALIAS  # last element of w
    assert step([item(0), item(0)]) == E_ALIAS  # one tensor twice
    assert step([item(0, g=FAKE)]) == E_ALIAS
    assert step([item(0, v=FAKE + 2 * MB + 4)]) == E_ALIAS
    assert step([item(0, state=1, vs=FAKE + 4 * MB + 12)]) == E_ALIAS  # 4 scales of 1000
    assert step([item(0), item(1, g=FAKE + 3 * MB + 400)]) == E_ALIAS  # g read where v is written
    assert step([item(0)], gs=ctypes.c_void_p(FAKE + 2 * MB)) == E_ALIAS
    # many tensors: the same check on a sorted list that does not fit the stack
    many = [item(k) for k in range(300)]
    many[299] = item(299, m=FAKE + 17 * 8 * MB + 3 * MB)
    assert step(many) == E_ALIAS


@needs_no_gpu
@pytest.mark.parametrize("count", [2, 3, 16, 64, 65, 66, 300])
@pytest.mark.parametrize("runs", [1, 2, 5, 31, 32, 33, 1000])
def test_step_alias_orders(count, runs):
    """One pair that overlaps is found, and no other, in whatever order the buffers lie."""
    rng = np.random.default_rng(count * 1000 + runs)
    order = np.arange(count)
    for part in np.array_split(order, min(runs, count)):
        rng.shuffle(part)  # in place, a view
    places = [item(int(k)) for k in order]
    rest = [p for p in places]
    assert step(rest) != E_ALIAS  # fails at the launch, for want of a device
    for name, of in (("w", "m"), ("g", "v"), ("v", "g")):
        i, j = int(rng.integers(count)), int(rng.integers(count - 1))
        j += j >= i
        bad = [p for p in places]
        bad[i] = item(int(order[i]), **{name: getattr(places[j], of) + 3996})
        assert step(bad) == E_ALIAS, (name, i, j)


@needs_no_gpu
def test_read_refusals():
    def read(n=1000, dtype=0, count=1, null=False, **at):
        a = {k: FAKE + j * MB for j, k in enumerate(("m", "v", "ms", "vs", "mo", "vo"))}
        a.update(at)
        s = (mao.Adamw8StateC * 1)(mao.Adamw8StateC(a["m"], a["v"], a["ms"], a["vs"], a["mo"],
                                                    a["vo"], n))
        return mao.load().mao_adamw8_read(count, None if null else s, dtype, None)

    assert read(null=True) == E_NULL
    assert read(count=0) == E_SHAPE
    assert read(n=-2) == E_SHAPE
    assert read(dtype=3) == E_DTYPE
    for k in ("m", "v", "ms", "vs", "mo", "vo"):
        assert read(**{k: None}) == E_NULL
    assert read(mo=FAKE + 4 * MB + 2) == E_LAYOUT
    assert read(ms=FAKE + 2 * MB + 2) == E_LAYOUT
    assert read(vo=FAKE + 4 * MB + 3996) == E_ALIAS
    assert read(mo=FAKE) == E_ALIAS


def test_binding_refusals():
    """Shapes, types and devices that the C call cannot see."""
    torch = pytest.importorskip("torch")
    w = torch.zeros(300)
    with pytest.raises(ValueError):
        mao.adamw_step_many([], 1, lr=1e-3)
    with pytest.raises(ValueError):
        mao.adamw8_read([])
    with pytest.raises(ValueError):  # host tensors
        mao.adamw_step_many([(w, w, w, w)], 1, lr=1e-3)
    with pytest.raises(TypeError):
        mao.adamw8_read([mao.adamw8_state(w)], dtype=torch.float16)
    m, ms, v, vs = mao.adamw8_state(torch.zeros((3, 100)))
    assert m.shape == v.shape == (3, 100) and ms.shape == vs.shape == (2,)
    assert m.dtype == v.dtype == torch.uint8 and ms.dtype == vs.dtype == torch.float32


@pytest.mark.parametrize("which,top,smallest", [("m", 1.875, 2.0 ** -17), ("v", 1.9375, 2.0 ** -18)])
def test_oracle_codes(which, top, smallest):
    """The values of all codes rise, by at most 1/8 (1/16) of themselves above the
    subnormals; the largest and the smallest are as the format says."""
    n = 128 if which == "m" else 256
    f = adam8.code_value(np.arange(n), which)
    assert f[0] == 0 and f[1] == smallest and f[-1] == top
    assert (np.diff(f) > 0).all()
    normal = np.arange(1 << adam8.MANTISSA[which], n)
    assert (np.diff(f[normal]) / f[normal][:-1] <= 0.5 ** adam8.MANTISSA[which]).all()


@pytest.mark.parametrize("which", ["m", "v"])
def test_oracle_round_trip_and_average(which):
    """What the codes stand for is stored without change; anything else as one of its two
    neighbours, and as itself on average over the steps. The average of N terms of the
    recurrence is off by its discrepancy, which for N = 512 is below 0.02 for both
    sequences (its largest gap between sorted points plus their unevenness, computed
    here)."""
    r = np.random.default_rng(5)
    top = 1.875 if which == "m" else 1.9375
    n = 128 if which == "m" else 256
    grid = adam8.code_value(np.arange(n), which)
    codes, scales = adam8.encode(grid, which, 9)
    assert (codes == np.arange(n)).all() and scales[0] == grid[-1] / top
    steps = 512
    pts = np.sort([adam8.dither(1, which, t)[0] for t in range(1, steps + 1)])
    i = np.arange(steps)
    disc = max(np.max((i + 1) / steps - pts), np.max(pts - i / steps))
    assert disc < 0.02
    x = np.concatenate([[1.0], np.exp(r.uniform(np.log(1e-3), 0.0, 60))])
    total = np.zeros_like(x)
    for t in range(1, steps + 1):
        c, s = adam8.encode(x, which, t)
        v = adam8.decode(c, s, which)
        step = np.maximum(2.0 ** np.floor(np.log2(x * top)), 2.0 ** -14) / top / 2 ** adam8.MANTISSA[which]
        assert (np.abs(v - x) <= step * (1 + 1e-12)).all()
        total += v
    # an element's dithers are the sequence shifted by its index: the same discrepancy times 2
    assert (np.abs(total / steps - x) <= 2 * disc * step).all()


def _fast_dither(n, which, t):
    """adam8.dither without Python's whole numbers: sums modulo 2^64, of which 2^32 divides."""
    a, b = adam8.DITHER[which]
    cut = 32 - 23 + adam8.MANTISSA[which]
    d = (np.arange(n, dtype=np.uint64) * np.uint64(a) + np.uint64(t * b % (1 << 32))) & np.uint64(0xFFFFFFFF)
    return (d >> np.uint64(cut)).astype(np.float64) * 0.5 ** (32 - cut)


def _store(x, which, t):
    """What a state that is to hold x holds, and its scales."""
    codes, scales = adam8.encode(x, which, t)
    return adam8.decode(codes, scales, which), scales


def test_oracle_dither_of_a_step_that_stands_still(monkeypatch):
    """A replayed graph repeats its t, and with it every element's dither d. A code then goes down
    only where (1 - beta1) of what is too much, in steps of the code, is above d: for 30% too much
    that is 0.1 0.3 / 1.3 of m, of which a step is 1/8 to 1/16, so 0.18 to 0.37. The dithers being
    equally spread, more than half of the elements stay where they are. As t advances all come
    down, to within a step of their value on average. What mao.h says of captured steps."""
    assert all((_fast_dither(777, k, 91) == adam8.dither(777, k, 91)).all() for k in "mv")
    monkeypatch.setattr(adam8, "dither", _fast_dither)
    g = np.exp(np.random.default_rng(1).uniform(np.log(0.05), np.log(0.7), 2048))
    g[::256] = 1.0  # holds its span's scale
    start = np.where(g == 1.0, 1.0, 1.3 * g)

    def last_steps(frozen):
        m, mean = start, np.zeros(g.size)
        for t in range(1, 301):
            m = _store(0.9 * m + 0.1 * g, "m", frozen or t)[0]
            mean += m / 150 if t > 150 else 0.0
        return mean

    assert (np.abs(last_steps(None) / g - 1) <= 1 / 8).all()
    for frozen in (4, 100):
        assert (last_steps(frozen) > 1.15 * g).mean() > 0.5


@pytest.mark.parametrize("spread", [0.5, 1.0, 3.0])
def test_oracle_second_moment_of_random_gradients(monkeypatch, spread):
    """beta2 = 0.999, gradients of magnitudes that differ within a span. The dither leaves r as it is
    on average, so r^2 gains the variance f (1 - f) step^2 of each rounding, where f step is at most
    what r moves in a step: (1 - beta2) / 2 |g^2 / v - 1| r, on average 0.97 times the first
    factor (normal g). A step is at most r / 16, so v gains 3e-5 of itself a step and 0.0303 over the
    1000 that it remembers. Elements whose r is below the smallest code, 2^-18 of the scale, hold
    that code instead."""
    monkeypatch.setattr(adam8, "dither", _fast_dither)
    n, steps, warm, b2 = 1024, 5000, 2500, 0.999
    rng = np.random.default_rng(3)
    s = np.exp(spread * rng.standard_normal(n))
    v, r, want, got = (np.zeros(n) for _ in range(4))
    for t in range(1, steps + 1):
        g = s * rng.standard_normal(n)
        v = b2 * v + (1 - b2) * g * g
        r, scales = _store(np.sqrt(b2 * r * r + (1 - b2) * g * g), "v", t)
        if t > warm:
            want += v
            got += r * r
    ratio, scale = got / want, np.repeat(scales, 256)
    whole = np.sqrt(v) >= 2.0 ** -13 * scale  # codes that have all their bits, and stay there
    assert whole.mean() > 0.5
    # four standard deviations of the mean
    assert abs(ratio[whole].mean() - 1 - 0.0303 / 2) < 0.0303 / 2 + 4 * ratio[whole].std() / whole.sum() ** 0.5
    assert (r >= 2.0 ** -18 * scale * (1 - 1e-12)).all()
    if spread == 3.0:
        low = np.sqrt(v) < 2.0 ** -20 * scale
        assert low.any() and (ratio[low] > 2).all()
