"""AdamW over many tensors with 32- and 8-bit states (GPU).

fp32 states: bit for bit what adamw_step gives. 8-bit states: against the float64 oracle,
starting from given codes. Error terms, in units of r = 2^-24 (half a step of fp32):
m = b1 m + (1 - b1) g is off by 3 r of its terms' magnitudes (the decoded m carries 1 of
them); v's terms are positive, so sqrt(v) is relatively off by at most 8 r (2 for the
square root's last place); the update by 16 r more (square root of ib2, sum, reciprocal,
product). A code is the floor of a place on the code axis: it may differ where the
place is nearer to a whole number than the value's relative error moves it, 2^(bits + 1) times
that error, plus as much for the scale and the dither's last bit; there, by one.
"""
import numpy as np
import pytest

from oracle import adam8
from tests.helpers import log

pytestmark = pytest.mark.gpu

R = 2.0 ** -24
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def _rand(seed, n, dtype="f32", scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g)) * scale
    return x.to(_types()[dtype]).cuda()


def _f32_item(seed, n, w="f32", g="f32"):
    return [_rand(seed, n, w), _rand(seed + 1, n, g), _rand(seed + 2, n, scale=0.3),
            _rand(seed + 3, n).square()]


SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 2047, 2048, 2049, 30000]


@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_equals_adamw_step(gpu_lib, w, g):
    """Every size in one call (more tensors than one launch holds), each with its own
    learning rate and decay."""
    import torch
    log(f"many fp32 states {w} {g}")
    sizes = SIZES * 9
    items = [_f32_item(10 * i, n, w, g) for i, n in enumerate(sizes)]
    want = [[t.clone() for t in it] for it in items]
    lr = [1e-3 * (1 + i % 5) for i in range(len(items))]
    wd = [0.1 * (i % 3) for i in range(len(items))]
    gpu_lib.adamw_step_many(items, 7, lr=lr, weight_decay=wd)
    for it, a, b in zip(want, lr, wd):
        gpu_lib.adamw_step(*it, 7, lr=a, weight_decay=b)
    torch.cuda.synchronize()
    for x, y in zip(items, want):
        for p, q in zip(x, y):
            assert torch.equal(p, q)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_back_to_back_tensors(gpu_lib, state):
    """Tensors at any element of flat buffers give what separate ones give, and nothing
    beside them is touched. A 2-D tensor is its elements in order; empty ones are skipped."""
    import torch
    log(f"back to back, {state}")
    sizes = [3, 2500, 0, 257, 8, 70000, 1]
    gap = 5
    total = sum(sizes) + gap * (len(sizes) + 1)
    spans = sum((n + 255) // 256 for n in sizes) + len(sizes) + 1

    def flat(n, dtype):
        return torch.full((n,), 77, dtype=dtype, device="cuda")

    bufs = {"w": flat(total, torch.bfloat16), "g": flat(total, torch.float32)}
    if state == "f32":
        bufs |= {"m": flat(total, torch.float32), "v": flat(total, torch.float32)}
    else:
        bufs |= {"m": flat(total, torch.uint8), "ms": flat(spans, torch.float32),
                 "v": flat(total, torch.uint8), "vs": flat(spans, torch.float32)}
    items, alone, at, sat, used = [], [], gap, 1, {k: [] for k in bufs}
    for i, n in enumerate(sizes):
        it, al = [], []
        for k, b in bufs.items():
            first, size = (sat, (n + 255) // 256) if k in ("ms", "vs") else (at, n)
            v = b[first:first + size]
            if k in ("ms", "vs"):
                v.copy_(_rand(40 * i + 1, size).abs() + 0.1)
            elif b.dtype == torch.uint8:
                v.copy_(torch.randint(1, 256, (size,)))
            else:
                v.copy_(_rand(40 * i + len(it), size).abs() if k == "v" else _rand(40 * i + len(it), size))
            used[k].append((first, size))
            it.append(v)
            al.append(v.clone())
        at += n + gap
        sat += (n + 255) // 256 + 1
        items.append(tuple(it))
        alone.append(tuple(al))
    items[1] = tuple(t.view(50, 50) if t.numel() == 2500 else t for t in items[1])
    gpu_lib.adamw_step_many(items, 3, **HP)
    for al in alone:
        if al[0].numel():
            gpu_lib.adamw_step_many([al], 3, **HP)
    torch.cuda.synchronize()
    for it, al in zip(items, alone):
        for x, y in zip(it, al):
            assert torch.equal(x.reshape(-1), y)
    for k, b in bufs.items():
        rest = torch.ones(b.numel(), dtype=torch.bool, device="cuda")
        for first, size in used[k]:
            rest[first:first + size] = False
        assert (b[rest] == 77).all(), k


def _state8(seed, n):
    """(m codes, m scales, v codes, v scales) with every code, zeros among them."""
    r = np.random.default_rng(seed)
    blocks = (n + 255) // 256
    return (r.integers(0, 256, n, dtype=np.uint8), (10.0 ** r.uniform(-6, 2, blocks)).astype(np.float32),
            r.integers(0, 256, n, dtype=np.uint8), (10.0 ** r.uniform(-6, 2, blocks)).astype(np.float32))


def _check_codes(got_codes, got_scales, x, rel, which, t):
    """Codes of x, whose computed value is relatively off by up to rel."""
    p, scales = adam8.places(x, which, t)
    rel = np.minimum(rel, 1.0)
    top_rel = np.array([rel[i:i + 256][np.argmax(np.abs(x[i:i + 256]))] for i in range(0, x.size, 256)])
    assert (np.abs(got_scales - scales) <= (top_rel + 4 * R) * scales).all()
    bits = adam8.MANTISSA[which]
    off = 2.0 ** (bits + 1) * (rel + np.repeat(top_rel, 256)[:x.size] + 8 * R) + 2.0 ** -19
    low, high = np.floor(p - off), np.floor(p + off)
    code = got_codes.astype(np.int64)
    if which == "m":
        assert ((code > 127) == (x < 0))[(x != 0) & (np.minimum(low, 127) > 0)].all()
        code = code & 127
        low, high = np.minimum(low, 127), np.minimum(high, 127)
    else:
        low = np.where(x > 0, np.clip(low, 1, 255), 0)
        high = np.where(x > 0, np.clip(high, 1, 255), 0)
    assert ((code >= low) & (code <= high)).all()
    # few places are that near to a border
    assert np.mean(low != high) < 0.01


@pytest.mark.parametrize("n", [1, 5, 8, 255, 256, 257, 2048, 2049, 70001])
@pytest.mark.parametrize("w,g,clip", [("f32", "f32", False), ("bf16", "bf16", True),
                                      ("bf16", "f32", False), ("f32", "bf16", True)])
def test_8bit_step(gpu_lib, n, w, g, clip):
    import torch
    log(f"8-bit step n={n} {w} {g}")
    mc, ms, vc, vs = _state8(n, n)
    W, G = _rand(n + 1, n, w), _rand(n + 2, n, g, 0.01)
    dev = [torch.from_numpy(a).cuda() for a in (mc, ms, vc, vs)]
    factor = torch.tensor(0.37, device="cuda") if clip else None
    t = 12
    w0, g0 = W.double().cpu().numpy(), G.double().cpu().numpy()
    gpu_lib.adamw_step_many([(W, G, *dev)], t, grad_scale=factor, **HP)
    b1, b2 = np.float64(np.float32(0.9)), np.float64(np.float32(0.95))
    lr, wd, eps = (np.float64(np.float32(x)) for x in (1e-2, 0.1, 1e-8))
    if clip:
        g0 = g0 * np.float64(np.float32(0.37))
    m0, r0 = adam8.decode(mc, ms, "m"), adam8.decode(vc, vs, "v")
    m = b1 * m0 + (1 - b1) * g0
    v = b2 * r0 ** 2 + (1 - b2) * g0 ** 2
    em = 4 * R * (np.abs(b1 * m0) + np.abs((1 - b1) * g0))
    rv = np.sqrt(v)
    den = rv / np.sqrt(1 - b2 ** t) + eps
    u = m / (1 - b1 ** t) / den
    eu = em / (1 - b1 ** t) / den + 24 * R * np.abs(u)
    want = w0 - lr * (wd * w0 + u)
    bound = lr * eu + 4 * R * (np.abs(w0) + lr * np.abs(u)) + 1e-37
    if w == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(want)
    got = W.double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all()
    out = [x.cpu().numpy() for x in dev]
    with np.errstate(divide="ignore", invalid="ignore"):
        rel = np.where(m != 0, em / np.abs(m), 0.0)
    _check_codes(out[0], out[1], m, rel, "m", t)
    _check_codes(out[2], out[3], rv, np.full(n, 8 * R), "v", t)
    # read back: the product of a code and a scale, one rounding each (v: squared)
    for dtype, half in ((torch.float32, R), (torch.bfloat16, 2.0 ** -8)):
        (rm, rvv), = gpu_lib.adamw8_read([tuple(dev)], dtype=dtype)
        em_ = adam8.decode(out[0], out[1], "m")
        ev_ = adam8.decode(out[2], out[3], "v") ** 2
        assert rm.dtype == rvv.dtype == dtype
        assert (np.abs(rm.double().cpu().numpy() - em_) <= (half + 2 * R) * np.abs(em_)).all()
        assert (np.abs(rvv.double().cpu().numpy() - ev_) <= (half + 6 * R) * np.abs(ev_)).all()


def test_8bit_from_zero_state_over_steps(gpu_lib):
    """From the zero state with a constant gradient, m / (1 - b1^t) stays g and v / (1 -
    b2^t) stays g^2 but for the codes: one step of theirs a step of the optimizer, averaged
    by (1 - b). m: b1 / (1 - b1) steps of 1/8 at the worst would be 1.1; the dither's
    signs alternate, so that the mean over 64 steps is within one code step."""
    import torch
    log("8-bit steps from zero")
    n, steps = 3000, 64
    G = _rand(3, n).abs().clamp(0.05, 20.0)
    W = torch.zeros(n, device="cuda")
    st = gpu_lib.adamw8_state(W)
    tm, tv = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for t in range(1, steps + 1):
        gpu_lib.adamw_step_many([(W, G, *st)], t, lr=0.0, beta1=0.9, beta2=0.95)
        (m, v), = gpu_lib.adamw8_read([st])
        tm += m / (1 - 0.9 ** t) / steps
        tv += v / (1 - 0.95 ** t) / steps
    assert ((tm - G).abs() <= G / 8).all()
    assert ((tv - G * G).abs() <= G * G / 8).all()


def test_8bit_zero_and_tiny_values(gpu_lib):
    """A span of zeros stays zero; magnitudes below the span's smallest code keep a
    denominator; a span below 2^-100 counts as zeros in m."""
    import torch
    log("8-bit zeros")
    n = 1024
    g = torch.zeros(n, device="cuda")
    g[256:512] = 1e-7
    g[300] = 100.0  # the others are 1e-9 of it
    g[512:768] = 1e-32
    w = torch.ones(n, device="cuda")
    st = gpu_lib.adamw8_state(w)
    gpu_lib.adamw_step_many([(w, g, *st)], 1, lr=1e-3)
    (m, v), = gpu_lib.adamw8_read([st])
    assert torch.isfinite(w).all() and torch.isfinite(m).all() and torch.isfinite(v).all()
    assert (m[:256] == 0).all() and (v[:256] == 0).all() and (w[:256] == 1).all()
    assert (v[256:512] > 0).all()  # never divided by eps alone
    assert (m[512:768] == 0).all() and st[1][2] == 0
    assert (m[768:] == 0).all()


def test_8bit_many(gpu_lib):
    """More tensors and rates than one launch holds, of both kinds of state: what single calls
    give, read back in one call too."""
    import torch
    log("many 8-bit")
    items = []
    for i in range(150):
        w = _rand(5 * i, SIZES[i % 11] + i // 11, ("f32", "bf16")[i % 2])
        g = _rand(5 * i + 1, w.numel(), ("f32", "bf16")[i // 2 % 2])
        items.append((w, g, *gpu_lib.adamw8_state(w)) if i % 5 else
                     (w, g, _rand(5 * i + 2, w.numel()), _rand(5 * i + 3, w.numel()).square()))
    want = [tuple(t.clone() for t in it) for it in items]
    lr = [1e-3 * (1 + i % 23) for i in range(len(items))]
    for t in (1, 2):
        gpu_lib.adamw_step_many(items, t, lr=lr, weight_decay=0.1)
        for it, a in zip(want, lr):
            gpu_lib.adamw_step_many([it], t, lr=a, weight_decay=0.1)
    torch.cuda.synchronize()
    for x, y in zip(items, want):
        for p, q in zip(x, y):
            assert torch.equal(p, q)
    states = [it[2:] for it in items if len(it) == 6]
    for got, st in zip(gpu_lib.adamw8_read(states), states):
        one, = gpu_lib.adamw8_read([st])
        assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_8bit_not_finite(gpu_lib, bad):
    """A span with a NaN or an infinity reads as NaN, all of it; the others do not."""
    import torch
    log(f"8-bit {bad}")
    n = 700
    w, g = torch.ones(n, device="cuda"), torch.full((n,), 0.1, device="cuda")
    g[300] = bad
    st = gpu_lib.adamw8_state(w)
    gpu_lib.adamw_step_many([(w, g, *st)], 1, lr=1e-3)
    (m, v), = gpu_lib.adamw8_read([st])
    for x in (m, v):
        assert torch.isnan(x[256:512]).all()
        assert torch.isfinite(x[:256]).all() and torch.isfinite(x[512:]).all()
    assert torch.isnan(w[300]) and torch.isfinite(w).sum() == n - 1


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_captured(gpu_lib, state):
    """A captured step, replayed with eager work between the replays, equals as many
    eager calls; two graphs of the same call do not disturb each other."""
    import torch
    log(f"captured {state}")
    sizes = [5000, 33, 256]

    def fresh():
        out = []
        for i, n in enumerate(sizes):
            w, g = _rand(i, n, "bf16"), _rand(i + 10, n, "bf16")
            s = gpu_lib.adamw8_state(w) if state == "8bit" else (torch.zeros(n, device="cuda"),
                                                                 torch.zeros(n, device="cuda"))
            out.append((w, g, *s))
        return out

    a, b, c = fresh(), fresh(), fresh()
    gpu_lib.adamw_step_many(fresh(), 4, **HP)
    torch.cuda.synchronize()
    graphs = []
    for items in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gpu_lib.adamw_step_many(items, 4, **HP)
        graphs.append(g)
    for k in range(3):
        graphs[0].replay()
        gpu_lib.adamw_step_many(c, 4, **HP)
        graphs[1].replay()
        torch.cuda.synchronize()
        for x, y, z in zip(a, b, c):
            for p, q, r in zip(x, y, z):
                assert torch.equal(p, r) and torch.equal(q, r)


def test_streams(gpu_lib):
    """Calls on two streams of their own at once give what one after the other gives."""
    import torch
    log("two streams")
    mk = lambda k: [(w := _rand(k, 100000, "bf16"), _rand(k + 1, 100000, "bf16"),
                     *gpu_lib.adamw8_state(w))]
    a, b, c, d = mk(1), mk(5), mk(1), mk(5)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for t in range(1, 6):
        with torch.cuda.stream(s1):
            gpu_lib.adamw_step_many(a, t, **HP)
        with torch.cuda.stream(s2):
            gpu_lib.adamw_step_many(b, t, **HP)
    torch.cuda.synchronize()
    for t in range(1, 6):
        gpu_lib.adamw_step_many(c, t, **HP)
        gpu_lib.adamw_step_many(d, t, **HP)
    for x, y in zip(a + b, c + d):
        for p, q in zip(x, y):
            assert torch.equal(p, q)


def test_refusals(gpu_lib):
    import torch
    log("refusals")
    lib = gpu_lib
    z = lambda n=300, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")
    w, g, m, v = z(), z(), z(), z()
    st = lib.adamw8_state(w)
    step = lambda items, t=1, **kw: lib.adamw_step_many(items, t, **{"lr": 1e-3, **kw})
    for items, error in (([(w, g, m)], ValueError), ([(w, g, m, v, z())], ValueError),
                         ([(w, z(299), m, v)], ValueError), ([(w, g, z(299), v)], ValueError),
                         ([(w, g, m, z(300, torch.bfloat16))], TypeError),
                         ([(z(300, torch.float16), g, m, v)], TypeError),
                         ([(w, z(300, torch.int32), m, v)], TypeError),
                         ([(w, g, m.cpu(), v)], ValueError), ([(w, g, m, None)], TypeError),
                         ([(w, g, z(600)[::2], v)], ValueError),
                         ([(w, g, st[0], st[1], st[2], z(1))], ValueError),
                         ([(w, g, st[0], z(2, torch.bfloat16), st[2], st[3])], TypeError),
                         ([(w, g, st[0].view(torch.int8), *st[1:])], TypeError),
                         ([w], ValueError)):
        with pytest.raises(error):
            step(items)
    for kw, error in ((dict(lr=[1e-3, 1e-3]), ValueError), (dict(lr="x"), TypeError),
                      (dict(weight_decay=[]), ValueError), (dict(grad_scale=z(2)), ValueError),
                      (dict(grad_scale=0.5), TypeError),
                      (dict(grad_scale=z(1, torch.bfloat16)), TypeError)):
        with pytest.raises(error):
            step([(w, g, m, v)], **kw)
    for items, kw, status in (([(w, g, m, v), (w, g, z(), z())], {}, 5), ([(w, w, m, v)], {}, 5),
                              ([(w, g, m, v)], dict(t=0), 6), ([(w, g, m, v)], dict(beta1=1.0), 6)):
        with pytest.raises(lib.MaoError) as e:
            step(items, **kw)
        assert e.value.status == status
    with pytest.raises(TypeError):
        step([(w, g, m, v)], t=1.5)
    with pytest.raises(ValueError):
        lib.adamw8_read([st], out=[(z(), z()), (z(), z())])
    with pytest.raises(ValueError):
        lib.adamw8_read([st], out=[(z(), z(299))])
    with pytest.raises(TypeError):
        lib.adamw8_read([st], out=[(z(), z(300, torch.bfloat16))])
    with pytest.raises(TypeError):
        lib.adamw8_read([st], out=[(z(300, torch.float16), z(300, torch.float16))])
    with pytest.raises(ValueError):
        lib.adamw8_read([st[:3]])
    for t in (w, g, m, v, *st):
        assert (t == 0).all()


def test_far_offsets(gpu_lib):
    """More than 2^32 elements: the last ones are stepped as a short tensor of the same
    values with the same place in their span."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GiB of free GPU memory are needed")
    log("far offsets")
    n = (1 << 32) + 256 * 3 + 5
    tail = 256 * 2 + 5
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    st = gpu_lib.adamw8_state(w)
    w[-tail:], g[-tail:] = _rand(1, tail, "bf16"), _rand(2, tail, "bf16")
    w1, g1 = w[-tail:].clone(), g[-tail:].clone()
    st1 = gpu_lib.adamw8_state(w1)
    # beta1 = beta2 = 0 keeps m = g, r = |g|; codes differ by the dither, the weights do not
    gpu_lib.adamw_step_many([(w, g, *st)], 2, lr=1e-2, beta1=0.0, beta2=0.0)
    gpu_lib.adamw_step_many([(w1, g1, *st1)], 2, lr=1e-2, beta1=0.0, beta2=0.0)
    torch.cuda.synchronize()
    assert torch.equal(w[-tail:], w1)
    assert torch.equal(st[1][-3:], st1[1]) and torch.equal(st[3][-3:], st1[3])
    assert (st[1][:-3] == 0).all() and not w[:1 << 20].any() and not w[-tail - 4096:-tail].any()
    (m1, v1), = gpu_lib.adamw8_read([(st[0][-tail:], st[1][-3:], st[2][-tail:], st[3][-3:])])
    gf = g1.float()
    assert ((m1 - gf).abs() <= torch.maximum(gf.abs() / 8, st[1][-3:].repeat_interleave(256)[:tail] * 2.0 ** -17) * 1.001).all()
    del w, g, st
    torch.cuda.empty_cache()


def _encode32(x, which, t):
    """Codes and scales of fp32 x, each operation rounded by itself (numpy's float32)."""
    f = np.float32
    n, k = x.size, adam8.MANTISSA[which]
    top = f(2.0 - 0.5 ** k)
    pad = np.zeros((n + 255) // 256 * 256, f)
    pad[:n] = np.abs(x)
    largest = pad.reshape(-1, 256).max(axis=1)
    live = largest >= f(2.0 ** -100)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(live, f(1) / largest * top, f(0))
    scales = np.where(live, largest * (f(1) / top), f(0))
    y = pad * np.repeat(inv, 256)
    drop = 23 - k
    a, b = adam8.DITHER[which]
    i = np.arange(pad.size, dtype=np.uint64)
    d = ((i * np.uint64(a) + np.uint64(t * b % (1 << 32))) & np.uint64(0xFFFFFFFF)) >> np.uint64(32 - drop)
    # the code's places with `drop` bits below them, cut off: a float's own bits, or, among the
    # subnormals, the multiple of 2^-37
    whole = y.view(np.int32).astype(np.int64) - (112 << 23)
    places = np.where(y < f(2.0 ** -14), np.floor(y.astype(np.float64) * 2.0 ** 37).astype(np.int64), whole)
    code = ((places + d.astype(np.int64)) >> drop)[:n]
    if which == "m":
        return np.minimum(code, 127) | np.where(np.signbit(x), 128, 0), scales
    return np.where((x > 0) & np.repeat(live, 256)[:n], np.clip(code, 1, 255), 0), scales


@pytest.mark.parametrize("g,clip", [("f32", False), ("bf16", True)])
def test_8bit_states_are_the_formulas(gpu_lib, g, clip):
    """States equal, bit for bit, what the formula's operations give, each rounded to fp32 by
    itself: a last bit more or less of m, r or a scale would be a whole code's step where a border
    is near, once in 2^20 elements, and w another one from the next step on."""
    import torch
    log(f"8-bit states as the formula {g}")
    f = np.float32
    n = 3_000_001
    mc, ms, vc, vs = _state8(5, n)
    ms[:3], vs[3:5] = (1e-30, 3e37, 2e-29), (1e-15, 1e-13)
    W, dev = _rand(1, n), [torch.from_numpy(a).cuda() for a in (mc, ms, vc, vs)]
    factor = torch.tensor(0.37, device="cuda") if clip else None
    m = adam8.decode(mc, np.ones(ms.size), "m").astype(f) * np.repeat(ms, 256)[:n]
    r = adam8.decode(vc, np.ones(vs.size), "v").astype(f) * np.repeat(vs, 256)[:n]
    b1, b2 = f(0.9), f(0.95)
    for t in (12, 13):
        G = _rand(t, n, g, 0.01)
        G[::1000] = 0.0
        x = G.float().cpu().numpy()
        if clip:
            x = x * f(0.37)
        gpu_lib.adamw_step_many([(W, G, *dev)], t, grad_scale=factor, **HP)
        m = b1 * m + (f(1) - b1) * x
        r = np.sqrt(b2 * (r * r) + (f(1) - b2) * x * x)
        assert m.dtype == r.dtype == f
        for k, (z, which) in enumerate(((m, "m"), (r, "v"))):
            codes, scales = _encode32(z, which, t)
            assert np.array_equal(dev[2 * k + 1].cpu().numpy(), scales), which
            got = dev[2 * k].cpu().numpy().astype(np.int64)
            assert (got != codes).sum() == 0, which
            value = adam8.decode(codes, np.ones(scales.size), which).astype(f)
            z[:] = value * np.repeat(scales, 256)[:n]
