"""The join between two blocks, forward and backward (GPU), against float64.

Errors are bounded element by element, in units of r = 2^-24 (half a step of fp32), with the
magnitudes of the terms (computed in float64). A sum over a row adds at most 16 terms in a
thread and 6 + 16 across the threads of a row, so a mean is off by 40 r of its terms'
magnitudes and by the mean of their own errors. Sums over rows: at most `rows` terms and 64 of
joins. A result in bf16 is off by 2^-8 of itself besides.
"""
import numpy as np
import pytest

from oracle import residual as ref
from tests.helpers import log

pytestmark = pytest.mark.gpu

R = 2.0 ** -24
EPS = 1e-5


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else R


def _dev(x, dtype):
    """x in rows padded to a multiple of 8 elements; the padding holds NaN."""
    import torch
    rows, cols = x.shape
    buf = torch.full((rows, (cols + 7) // 8 * 8), float("nan"),
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    buf[:, :cols] = torch.from_numpy(np.asarray(x, np.float32)).cuda()
    return buf[:, :cols]


def _vec(x, dtype="f32"):
    import torch
    v = torch.from_numpy(np.asarray(x, np.float32)).cuda()
    return v.bfloat16() if dtype == "bf16" else v


def _host(t):
    return t.double().cpu().numpy()


class Case:
    """Inputs of both directions, on the device and as the float64 values they hold."""

    def __init__(self, seed, rows, cols, xt, bt, post, pre, gate, pt="f32"):
        r = np.random.default_rng(seed)
        scale = np.exp(0.5 * r.standard_normal((rows, 1)))
        self.rows, self.cols, self.xt, self.bt = rows, cols, xt, bt
        self.post, self.pre, self.gate = post, pre, gate
        self.xs, self.bs = 0.75, -1.5
        x = r.standard_normal((rows, cols)) * scale + 0.3
        b = r.standard_normal((rows, cols)) * scale - 0.2
        x[1::4] = 0.0  # padding rows
        b[2::4] = 0.0
        self.X, self.B = _dev(x, xt), _dev(b, bt)
        self.dH = _dev(1e-2 * r.standard_normal((rows, cols)), bt)
        self.dR = _dev(1e-2 * r.standard_normal((rows, cols)), xt)
        kw = {}
        for name, kind in (("post", post), ("pre", pre)):
            kw[name] = kind
            if kind != "none":
                kw[name + "_gamma"] = _vec(1 + 0.3 * r.standard_normal(cols), pt)
            if kind == "layer":
                kw[name + "_beta"] = _vec(0.2 * r.standard_normal(cols), pt)
        if gate == "vector":
            kw["gate"] = _vec(0.5 + 0.5 * r.standard_normal(cols), pt)
        if gate == "matrix":
            kw["gate"] = _dev(0.5 + 0.5 * r.standard_normal((rows, cols)), bt)
        self.kw = dict(kw, x_scale=self.xs, b_scale=self.bs)
        h = lambda k, default: _host(kw[k]) if k in kw else default
        self.n1 = (post, h("post_gamma", 1.0), h("post_beta", 0.0))
        self.n2 = (pre, h("pre_gamma", 1.0), h("pre_beta", 0.0))
        self.g = h("gate", 1.0)

    def back_kw(self):
        return {k: v for k, v in self.kw.items() if k != "pre_beta"}


def _mean(z):
    return np.abs(z).mean(axis=1, keepdims=True)


def _norm_bound(z, ez, norm, eps=EPS):
    """Error of N(z), of the mean and of rstd for a z with errors ez."""
    kind, gamma, beta = norm
    if kind == "none":
        return ez, 0.0, 0.0
    em = 40 * R * _mean(z) + ez.mean(axis=1, keepdims=True) if kind == "layer" else 0.0 * z[:, :1]
    mean = z.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    d = z - mean
    ed = ez + em + R * np.abs(d)
    var = (d * d).mean(axis=1, keepdims=True) + eps
    s = var ** -0.5
    es = ((np.abs(d) * ed + ed * ed).mean(axis=1, keepdims=True) / var + 50 * R)  # relative
    y = np.abs(d * s * gamma)
    return np.abs(gamma) * s * ed + y * es + 4 * R * (y + np.abs(beta)), em[:, 0], (s * es)[:, 0]


def _check_forward(c, got):
    x, b = _host(c.X), _host(c.B)
    r, h, st = ref.forward(x, b, c.g, c.xs, c.bs, c.n1, c.n2, EPS)
    eu, em1, es1 = _norm_bound(b, np.zeros_like(b), c.n1)
    w = r - c.xs * x
    er = np.abs(c.bs * c.g) * eu + 4 * R * (np.abs(c.xs * x) + np.abs(w))
    assert (np.abs(_host(got[0]) - r) <= er + _half(c.xt) * np.abs(r)).all()
    s = _host(got[2])
    for k, (want, bound) in enumerate(((st[0], em1), (st[1], es1))):
        assert (np.abs(s[:, k] - want) <= bound + R * np.abs(want)).all()
    if c.pre == "none":
        assert got[1] is None and (s[:, 2] == 0).all() and (s[:, 3] == 1).all()
        return
    eh, em2, es2 = _norm_bound(r, er, c.n2)
    assert (np.abs(_host(got[1]) - h) <= eh + _half(c.bt) * np.abs(h)).all()
    for k, (want, bound) in enumerate(((st[2], em2), (st[3], es2))):
        assert (np.abs(s[:, 2 + k] - want) <= bound + R * np.abs(want)).all()


def _check_backward(c, got, Rr, stats, dr=True):
    b, r = _host(c.B), None if Rr is None else _host(Rr)
    s = _host(stats)
    st = (s[:, 0], s[:, 1], s[:, 2], s[:, 3])
    d0 = _host(c.dR) if dr else None
    dh = _host(c.dH) if c.pre != "none" else None
    dx, db, dg, g1, b1, g2, b2 = ref.backward(dh, d0, b, r, st, c.g, c.xs, c.bs, c.n1, c.n2)

    def through(dy, e, z, norm, mean, rstd):
        """Error of the gradient through a norm for a dy with errors e, and |dy xh|, its error."""
        kind, gamma, _ = norm
        if kind == "none":
            return e, np.abs(dy * z), e * np.abs(z)
        xh = np.abs((z - mean[:, None]) * rstd[:, None])
        exh = 2 * R * xh + R * np.abs(z - mean[:, None]) * rstd[:, None]
        q, eq = np.abs(dy * gamma), np.abs(gamma) * e + R * np.abs(dy * gamma)
        m0 = eq.mean(axis=1, keepdims=True) + 42 * R * _mean(q)
        m1 = (eq * xh + q * exh).mean(axis=1, keepdims=True) + 44 * R * _mean(q * xh)
        total = eq + m0 + xh * m1 + (exh + 4 * R * xh) * _mean(q * xh) + 4 * R * (q + _mean(q))
        return rstd[:, None] * total, np.abs(dy) * xh, e * xh + np.abs(dy) * exh

    zero = np.zeros_like(b)
    ed = zero
    if c.pre != "none":
        ed, t2, et2 = through(dh, zero, r, c.n2, st[2], st[3])
    d = dx / c.xs
    ed = ed + 4 * R * (np.abs(d) + (np.abs(d0) if dr else 0.0))
    half_x, half_b = _half(c.xt), _half(c.bt)
    assert (np.abs(_host(got.dX) - dx) <= abs(c.xs) * ed + (half_x + 2 * R) * np.abs(dx)).all()
    du = c.bs * c.g * d
    edu = np.abs(c.bs * c.g) * ed + 4 * R * np.abs(du)
    eb, t1, et1 = through(du, edu, b, c.n1, st[0], st[1])
    assert (np.abs(_host(got.dB) - db) <= eb + (half_b + 4 * R) * np.abs(db)).all()
    chain = (c.rows + 64) * R

    def column(x, want, term, err):
        assert (np.abs(_host(x) - want) <= (err + (chain + 6 * R) * term).sum(axis=0)).all()

    if c.post != "none":
        column(got.dpost_gamma, g1, t1, et1)
    else:
        assert got.dpost_gamma is None
    if c.post == "layer":
        column(got.dpost_beta, b1, np.abs(du), edu)
    else:
        assert got.dpost_beta is None
    if c.pre != "none":
        column(got.dpre_gamma, g2, t2, et2)
    else:
        assert got.dpre_gamma is None
    if c.pre == "layer":
        column(got.dpre_beta, b2, np.abs(dh), zero)
    else:
        assert got.dpre_beta is None
    # the gate's gradient, term by term: bs dr (xh gamma + beta)
    kind, gamma, beta = c.n1
    xh = b if kind == "none" else (b - st[0][:, None]) * st[1][:, None]
    terms = np.abs(c.bs * d) * (np.abs(xh * gamma) + np.abs(beta))
    eterm = np.abs(c.bs) * ed * (np.abs(xh * gamma) + np.abs(beta)) + 8 * R * terms
    if c.gate == "vector":
        column(got.dgate, dg.sum(axis=0), terms, eterm)
    elif c.gate == "matrix":
        assert got.dgate.dtype == c.B.dtype
        assert (np.abs(_host(got.dgate) - dg) <= eterm + half_b * np.abs(dg)).all()
    else:
        assert got.dgate is None


def _run(lib, c, dr=True):
    import torch
    got = lib.residual_norm(c.X, c.B, eps=EPS, **c.kw)
    assert got[0].dtype == c.X.dtype and (got[1] is None or got[1].dtype == c.B.dtype)
    _check_forward(c, got)
    none = c.pre == "none"
    back = lib.residual_norm_backward(None if none else c.dH, c.dR if dr else None, c.B,
                                      None if none else got[0], got[2], **c.back_kw())
    _check_backward(c, back, None if none else got[0], got[2], dr)
    again = lib.residual_norm_backward(None if none else c.dH, c.dR if dr else None, c.B,
                                       None if none else got[0], got[2], **c.back_kw())
    for p, q in zip(back, again):
        assert (p is None and q is None) or torch.equal(p, q)
    return got, back


KINDS = ["none", "layer", "rms"]


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("gate", ["none", "vector", "matrix"])
def test_kinds(gpu_lib, post, pre, gate):
    """Every pair of norms with every gate, in all types, odd sizes."""
    log(f"kinds {post} {pre} {gate}")
    for k, (xt, bt) in enumerate((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32"))):
        _run(gpu_lib, Case(k, 41, 301, xt, bt, post, pre, gate, "bf16" if k == 1 else "f32"))
        _run(gpu_lib, Case(9 + k, 5, 1540, xt, bt, post, pre, gate), dr=pre == "none")


COLS = [1, 2, 3, 4, 5, 8, 64, 255, 256, 257, 511, 513, 768, 770, 1000, 1025, 1536, 2048, 2049, 2560, 2563,
        4096, 4100, 5120, 6144, 6145, 8192, 8193, 16384]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_widths(gpu_lib, cols, types):
    for rows in (1, 3, 67) + ((2100,) if cols <= 257 else (700,) if cols <= 1536 else ()):
        log(f"width {rows} x {cols} {types}")
        gate = ("none", "vector", "matrix")[(cols + rows) % 3]
        _run(gpu_lib, Case(cols + rows, rows, cols, *types, "layer", "layer", gate))
        if rows < 100:
            _run(gpu_lib, Case(cols + rows, rows, cols, *types, "rms", "rms", gate), dr=rows > 1)


def test_parameters_left_out(gpu_lib):
    """gamma and beta default to 1 and 0; scales to 1; without statistics and sums."""
    import torch
    log("defaults")
    c = Case(3, 9, 72, "f32", "f32", "layer", "rms", "none")
    one, zero = torch.ones(72, device="cuda"), torch.zeros(72, device="cuda")
    r, h, st = gpu_lib.residual_norm(c.X, c.B, post="layer")
    r2, h2, st2 = gpu_lib.residual_norm(c.X, c.B, post="layer", post_gamma=one, post_beta=zero, pre="rms",
                                        pre_gamma=one, x_scale=1.0, b_scale=1.0, eps=1e-5, gate=one)
    assert torch.equal(r, r2) and torch.equal(h, h2) and torch.equal(st, st2)
    r3, h3, none = gpu_lib.residual_norm(c.X, c.B, post="layer", stats=False)
    assert none is None and torch.equal(r3, r) and torch.equal(h3, h)
    a = gpu_lib.residual_norm_backward(c.dH, c.dR, c.B, r, st, post="layer")
    b = gpu_lib.residual_norm_backward(c.dH, c.dR, c.B, r, st, post="layer", sums=False)
    assert torch.equal(a.dX, b.dX) and torch.equal(a.dB, b.dB)
    assert b[2:] == (None,) * 5 and a.dpost_gamma is not None and a.dpre_beta is None


@pytest.mark.parametrize("rows,cols", [(2300, 601), (1100, 2501), (1100, 5121), (600, 7003), (600, 9001)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_wide_rows_in_turn(gpu_lib, rows, cols, types):
    """More rows than workgroups at once, each with several runs a thread."""
    log(f"wide rows {rows} x {cols} {types}")
    _run(gpu_lib, Case(3, rows, cols, *types, "layer", "rms", "vector"))


@pytest.mark.parametrize("cols", [30, 1030, 8200])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_in_place_and_views(gpu_lib, cols, types):
    """The stream updated in place, dX in place of dR, and views of wider buffers give the same
    and leave the rest alone."""
    import torch
    log(f"in place {cols} {types}")
    c = Case(cols, 7, cols, *types, "layer", "layer", "matrix")
    want, back = _run(gpu_lib, c)
    ld = (cols + 7) // 8 * 8 + 16

    def wide(t):
        buf = torch.full((9, ld), 3.0, dtype=t.dtype, device="cuda")
        v = buf[1:8, 8:8 + cols]
        v.copy_(t)
        return buf, v

    def untouched(buf):
        keep = buf.clone()
        keep[1:8, 8:8 + cols] = 3.0
        return bool((keep == 3.0).all())

    xb, x = wide(c.X)
    bb, b = wide(c.B)
    hb, h = wide(c.B)
    gb, g = wide(c.kw["gate"])
    kw = {**c.kw, "gate": g}
    got = gpu_lib.residual_norm(x, b, eps=EPS, out=x, h=h, **kw)
    assert got[0].data_ptr() == x.data_ptr() and got[1].data_ptr() == h.data_ptr()
    assert torch.equal(x, want[0]) and torch.equal(h, want[1]) and torch.equal(got[2], want[2])
    db, d = wide(c.dR)
    kw = {k: v for k, v in kw.items() if k != "pre_beta"}
    o = gpu_lib.residual_norm_backward(c.dH, d, b, x, got[2], out=d, **kw)
    assert o.dX.data_ptr() == d.data_ptr()
    for p, q in zip(o, back):
        assert torch.equal(p, q)
    for buf in (xb, bb, hb, gb, db):
        assert untouched(buf)


def test_special_rows(gpu_lib):
    """A NaN or an infinity stays in its row, forward and backward; rows of zeros stay finite."""
    import torch
    log("special rows")
    c = Case(8, 70, 520, "bf16", "bf16", "rms", "layer", "vector")
    c.X[3, 100], c.B[6, 5], c.B[9, 0] = float("nan"), float("inf"), float("nan")
    r, h, st = gpu_lib.residual_norm(c.X, c.B, **c.kw)
    bad = [3, 6, 9]
    good = [i for i in range(70) if i not in bad]
    assert torch.isfinite(r[good].float()).all() and torch.isfinite(h[good].float()).all()
    assert torch.isfinite(st[good]).all() and not torch.isfinite(h[bad].float()).all(dim=1).any()
    g = gpu_lib.residual_norm_backward(c.dH, c.dR, c.B, r, st, **c.back_kw())
    assert torch.isfinite(g.dX[good].float()).all() and torch.isfinite(g.dB[good].float()).all()
    assert not torch.isfinite(g.dpre_gamma).all()


def test_captured(gpu_lib):
    """Two graphs with workspaces, eager calls of a larger workspace between the replays, new
    inputs for every replay."""
    import torch
    log("captured")
    cases = [Case(1, 600, 1536, "bf16", "bf16", "layer", "layer", "vector"),
             Case(2, 300, 2000, "f32", "bf16", "rms", "rms", "matrix")]
    big = Case(3, 700, 8192, "bf16", "bf16", "rms", "rms", "none")

    def call(c):
        r, h, st = gpu_lib.residual_norm(c.X, c.B, **c.kw)
        return (r, h, st, *gpu_lib.residual_norm_backward(c.dH, c.dR, c.B, r, st, **c.back_kw()))

    for c in cases:
        call(c)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c))
        graphs.append(g)
    for k in range(3):
        for c in cases:
            c.X.add_(0.25)
            c.dH.mul_(1.5)
        graphs[0].replay()
        call(big)
        graphs[1].replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            for p, q in zip(o, call(c)):
                assert (p is None and q is None) or torch.equal(p, q)


def test_two_streams(gpu_lib):
    import torch
    log("two streams")
    cases = [Case(k, 500, 1536, "bf16", "bf16", "rms", "rms", "vector") for k in (1, 2)]

    def call(c):
        r, h, st = gpu_lib.residual_norm(c.X, c.B, **c.kw)
        return (r, h, st, *gpu_lib.residual_norm_backward(c.dH, c.dR, c.B, r, st, **c.back_kw()))

    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for k in range(8):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                got[i].append(call(cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            for p, q in zip(o, want[i]):
                assert (p is None and q is None) or torch.equal(p, q)


def test_far_offsets(gpu_lib):
    """Rows whose offsets pass 2^32 elements."""
    import torch
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GiB of free GPU memory are needed")
    log("far offsets")
    rows, ld, cols = 70001, 65536, 72
    x, b, dh = (torch.randn((rows, cols), device="cuda").bfloat16() for _ in range(3))
    bufs = [torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    fx, fb, fo = (t[:, :cols] for t in bufs)
    fx.copy_(x)
    fb.copy_(b)
    kw = dict(post="layer", pre="layer")
    want = gpu_lib.residual_norm(x, b, **kw)
    got = gpu_lib.residual_norm(fx, fb, out=fo, **kw)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    w = gpu_lib.residual_norm_backward(dh, x, b, want[0], want[2], **kw)
    g = gpu_lib.residual_norm_backward(dh, fx, fb, fo, want[2], out=fx, **kw)
    for p, q in zip(g, w):
        assert (p is None and q is None) or torch.equal(p, q)
    del bufs, fx, fb, fo
    torch.cuda.empty_cache()


def test_refusals(gpu_lib):
    import torch
    log("refusals")
    lib = gpu_lib
    x, b, v = torch.randn((4, 64), device="cuda"), torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    r, h, st = lib.residual_norm(x, b)
    E = lib.MaoError
    for call, error in (
            (lambda: lib.residual_norm(x, b[:3]), E),
            (lambda: lib.residual_norm(x, b, gate=v[:32]), ValueError),
            (lambda: lib.residual_norm(x, b, gate=v.half()), TypeError),
            (lambda: lib.residual_norm(x, b, gate=b.bfloat16()), E),
            (lambda: lib.residual_norm(x, b, gate=1.0), TypeError),
            (lambda: lib.residual_norm(x, b, post_gamma=v), E),
            (lambda: lib.residual_norm(x, b, pre_beta=v), E),
            (lambda: lib.residual_norm(x, b, pre="layer", pre_gamma=v, pre_beta=v.bfloat16()), TypeError),
            (lambda: lib.residual_norm(x, b, eps=0.0), E),
            (lambda: lib.residual_norm(x, b, x_scale=float("nan")), E),
            (lambda: lib.residual_norm(x, b, x_scale="1"), TypeError),
            (lambda: lib.residual_norm(x.half(), b), TypeError),
            (lambda: lib.residual_norm(x.cpu(), b), ValueError),
            (lambda: lib.residual_norm(x, b.cpu()), ValueError),
            (lambda: lib.residual_norm(x, b, out=b), E),
            (lambda: lib.residual_norm(x, b, out=x.bfloat16()), E),
            (lambda: lib.residual_norm(x, b, pre="none", h=b.clone()), E),
            (lambda: lib.residual_norm(x.clone().requires_grad_(True), b), RuntimeError),
            (lambda: lib.residual_norm_backward(None, x, b, r, st), E),
            (lambda: lib.residual_norm_backward(h, x, b, None, st), E),
            (lambda: lib.residual_norm_backward(None, None, b, None, st, pre="none"), ValueError),
            (lambda: lib.residual_norm_backward(h, x, b, r, st[:3]), ValueError),
            (lambda: lib.residual_norm_backward(h, x, b, r, st.double()), TypeError),
            (lambda: lib.residual_norm_backward(h, x, b, r, None), TypeError),
            (lambda: lib.residual_norm_backward(h, x.bfloat16(), b, r, st), E),
            (lambda: lib.residual_norm_backward(h, x, b, r, st, out=r), E)):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("cols", [30, 301, 1540, 5000, 9000])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("gate", ["none", "vector", "matrix"])
def test_not_finite_without_a_norm_of_the_block(gpu_lib, cols, types, gate):
    """Without a norm of the block's output its gradient is made element by element: a NaN or an
    infinity in one leaves all the others alone."""
    import torch
    log(f"not finite, no post norm {cols} {types} {gate}")
    for pre in ("none", "rms"):
        c = Case(cols, 5, cols, *types, "none", pre, gate)
        r, _, st = gpu_lib.residual_norm(c.X, c.B, **c.kw)
        call = lambda: gpu_lib.residual_norm_backward(  # noqa: E731
            None if pre == "none" else c.dH, c.dR, c.B, None if pre == "none" else r, st, sums=False,
            **c.back_kw())
        want = call()
        at = torch.zeros((5, cols), dtype=torch.bool, device="cuda")
        for k, bad in enumerate((float("inf"), -float("inf"), float("nan"))):
            c.dR[k, 7 * k + 8] = bad
            at[k, 7 * k + 8] = True
        got = call()
        for p, q in ((got.dX, want.dX), (got.dB, want.dB)) + (((got.dgate, want.dgate),) if gate == "matrix" else ()):
            assert torch.equal(p[~at], q[~at])
            assert not torch.isfinite(p[at].float()).any()


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_infinite_gradient_of_a_gate_vector(gpu_lib, post):
    """One infinite dR makes its column's gate gradient infinite, of the sign that the formula gives;
    the other columns keep theirs."""
    import torch
    log(f"infinite gate gradient {post}")
    c = Case(5, 40, 301, "f32", "f32", post, "none", "vector")
    c.kw.pop("post_beta", None)  # no offset: the gradient is the sum of dR xh gamma alone
    r, _, st = gpu_lib.residual_norm(c.X, c.B, **c.kw)
    want = gpu_lib.residual_norm_backward(None, c.dR, c.B, None, st, **c.back_kw()).dgate
    c.dR[7, 33] = float("inf")
    got = gpu_lib.residual_norm_backward(None, c.dR, c.B, None, st, **c.back_kw()).dgate
    xh = (c.B[7, 33] - st[7, 0]) * st[7, 1] * (c.kw["post_gamma"][33] if post != "none" else 1.0)
    assert got[33] == c.bs * xh * float("inf")
    keep = torch.arange(301, device="cuda") != 33
    assert torch.equal(got[keep], want[keep])
