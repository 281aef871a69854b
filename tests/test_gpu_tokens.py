"""Log probabilities of tokens, their alternatives and gradients (GPU), against float64.

Error terms, in units of r = 2^-24 (half a step of fp32). y = x - M is off by r |y|. A term
e^y of the sum S: |y| for that, |y| and |y| for the product with log2 e and its constant, 2
for the exponential's last place: 3 |y| + 2; those that count have |y| below 20. The sum
adds at most 100 terms in a row anywhere (a thread's, then two wavefront sums), so that S is
off by 170 r relatively. Its logarithm then by 170 r + 2 r |log S|. T's terms have one sign:
the same and |y|'s own error, 180 r. A probability e^(y - log S) by (6 |y| + 2 log S + 180) r,
and by 2^-126, where the exponential's result is no longer a normal number.
"""
import numpy as np
import pytest

from oracle import tokens as ref
from tests.helpers import log

# infinities are compared apart, differences of them are NaN and left out
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value")]

R = 2.0 ** -24


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else R


def _dev(x, dtype, pad=float("nan")):
    """x in rows padded to a multiple of 8 elements; the padding holds NaN."""
    import torch
    rows, cols = x.shape
    buf = torch.full((rows, (cols + 7) // 8 * 8), pad,
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    buf[:, :cols] = torch.from_numpy(np.asarray(x, np.float32)).cuda()
    return buf[:, :cols]


def _host(t):
    return t.double().cpu().numpy()


def _logits(seed, rows, vocab, masked=0):
    r = np.random.default_rng(seed)
    x = 2.5 * r.standard_normal((rows, vocab)) + 2 * r.standard_normal((1, vocab))
    if masked:
        x[:, r.permutation(vocab)[:masked]] = -np.inf
    t = r.integers(0, vocab, rows)
    t[2::5] = -1
    return x, t


def _targets(t):
    import torch
    return torch.from_numpy(np.asarray(t, np.int64)).cuda()


def _check_forward(lib, x, t, dtype, top=0, entropy=True):
    X = _dev(x, dtype)
    x = _host(X)
    got = lib.token_logprobs(X, _targets(t), top=top, entropy=entropy)
    lp, ent, big, log_s, logp = ref.forward(x, t)
    y = np.where(np.isfinite(lp), lp + log_s, 0.0)
    err = (170 + np.abs(y) + 2 * np.abs(log_s) + np.abs(y + log_s)) * R + 2 * R * np.abs(log_s)
    assert np.array_equal(np.isfinite(_host(got.logprob)), np.isfinite(lp))
    ok = np.isfinite(lp)
    assert (np.abs(_host(got.logprob) - lp)[ok] <= err[ok]).all()
    st = _host(got.stats)
    assert np.array_equal(st[:, 0], big)
    assert (np.abs(st[:, 1] - log_s) <= (170 + 2 * np.abs(log_s)) * R).all()
    if entropy:
        ts = np.abs(log_s - ent)  # |T / S|
        assert (np.abs(_host(got.entropy) - ent) <= (170 + 2 * np.abs(log_s) + 400 * ts + 2 * ent) * R).all()
    else:
        assert got.entropy is None
    if top:
        ids = ref.top(x, top)
        assert np.array_equal(got.top_ids.cpu().numpy(), ids)
        want = np.take_along_axis(logp, ids, axis=1)
        tl = _host(got.top_logprobs)
        assert np.array_equal(np.isinf(tl), np.isinf(want))
        fin = np.isfinite(want)
        bound = (170 + 2 * np.abs(log_s)[:, None] + 2 * np.abs(np.where(fin, want, 0)) + 2 * np.abs(log_s)[:, None]) * R
        assert (np.abs(np.where(fin, tl - want, 0)) <= bound).all()
    else:
        assert got.top_ids is None and got.top_logprobs is None
    return got


VOCABS = [1, 2, 7, 8, 9, 63, 200, 1000, 1024, 1025, 4099, 8192, 8193, 20001, 50301, 65537, 140000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_forward(gpu_lib, vocab, dtype):
    """One row, a few, and more than a thousand short ones."""
    for rows in (1, 7) + ((1300,) if vocab <= 1025 else ()):
        log(f"forward {rows} x {vocab} {dtype}")
        x, t = _logits(vocab + rows, rows, vocab, masked=vocab // 5)
        for top in {0, min(vocab, 1), min(vocab, 5), min(vocab, 32)}:
            _check_forward(gpu_lib, x, t, dtype, top)
    _check_forward(gpu_lib, x, t, dtype, 0, entropy=False)
    _check_forward(gpu_lib, x, t, dtype, min(vocab, 3), entropy=False)


def test_forward_whole_rows_of_a_batch(gpu_lib):
    """Many rows of 256 threads and of 512, of several blocks."""
    log("forward, rows of a batch")
    for rows, vocab in ((520, 9001), (300, 70003)):
        x, t = _logits(3, rows, vocab)
        _check_forward(gpu_lib, x, t, "bf16", 20)
        _check_forward(gpu_lib, x, t, "f32", 32)


@pytest.mark.parametrize("vocab", [40, 1000, 9000, 50304])
@pytest.mark.parametrize("rows", [1, 600])
def test_alternatives_of_awkward_rows(gpu_lib, rows, vocab):
    """Ties (also of -0 and 0), flat rows, masks that leave few or neighbouring tokens, rows in
    order: exact tokens, in order."""
    if rows * vocab > 6_000_000:
        rows = 6_000_000 // vocab
    log(f"alternatives {rows} x {vocab}")
    r = np.random.default_rng(vocab + rows)
    kinds = []
    flat = np.full(vocab, 1.5)
    few = np.full(vocab, -np.inf)
    few[[vocab // 2, 1, vocab - 1]] = [0.5, 2.0, 0.5]
    block = np.full(vocab, -np.inf)
    width = min(vocab, 3900)
    block[vocab - width:] = r.standard_normal(width)
    zeros = np.where(r.random(vocab) < 0.5, -0.0, 0.0)
    steps = r.integers(0, 4, vocab).astype(np.float64)
    low = np.full(vocab, -3.3895313892515355e38)  # the lowest bf16
    low[vocab // 3] = 0.0
    kinds = [flat, few, block, zeros, steps, low, np.arange(vocab) / 64.0, -np.arange(vocab) / 64.0]
    x = np.stack([kinds[i % len(kinds)] for i in range(max(rows, len(kinds)))])
    t = r.integers(0, vocab, len(x))
    pieces = [x] if rows > 1 else [x[i:i + 1] for i in range(len(kinds))]
    for k, z in enumerate(pieces):
        for dtype in ("bf16", "f32"):
            X = _dev(z, dtype)
            tt = t[k:k + 1] if rows == 1 else t
            got = gpu_lib.token_logprobs(X, _targets(tt), top=32)
            assert np.array_equal(got.top_ids.cpu().numpy(), ref.top(_host(X), 32))
            logp = ref.forward(_host(X), tt)[4]
            want = np.take_along_axis(logp, got.top_ids.cpu().numpy(), axis=1)
            tl = _host(got.top_logprobs)
            assert np.array_equal(np.isinf(tl), np.isinf(want))
            fin = np.isfinite(want)
            assert (np.abs(np.where(fin, tl - want, 0)) <= (400 + 4 * np.abs(np.where(fin, want, 0))) * R).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [100, 9000, 70000])
def test_rows_of_special_values(gpu_lib, vocab, dtype):
    """Nothing but masked logits; NaN; +inf; the type's lowest value everywhere; logits far
    from 0; targets that are masked or outside the vocabulary. Other rows are not touched
    by them."""
    log(f"special rows {vocab} {dtype}")
    x, _ = _logits(1, 9, vocab)
    x = x.astype(np.float32).astype(np.float64)
    x[0] = -np.inf
    x[1, vocab // 2] = np.nan
    x[2, vocab - 1] = np.inf
    x[3] = -3.3895313892515355e38
    x[4] += 4096.0
    x[5, 3] = -np.inf
    x[7] = -np.inf
    x[7, 1] = 2.0
    t = np.array([3, 3, 3, 3, 3, 3, vocab, 1, -1])
    X = _dev(x, dtype)
    x = _host(X)
    got = gpu_lib.token_logprobs(X, _targets(t), top=4)
    lp, ent, st = _host(got.logprob), _host(got.entropy), _host(got.stats)
    ids, tl = got.top_ids.cpu().numpy(), _host(got.top_logprobs)
    assert lp[0] == -np.inf and ent[0] == 0 and st[0].sum() == -np.inf
    assert ids[0].tolist() == [0, 1, 2, 3] and (tl[0] == -np.inf).all()
    for i in (1, 2):
        assert np.isnan([lp[i], ent[i], *tl[i]]).all() and (ids[i] == -1).all()
    n = np.log(vocab)
    assert abs(lp[3] + n) < 200 * R * n and abs(ent[3] - n) < 200 * R * n
    assert lp[5] == -np.inf and np.isnan(lp[6]) and lp[8] == 0
    assert lp[7] == 0 and ent[7] == 0 and ids[7].tolist() == [1, 0, 2, 3]
    keep = [4, 5, 6, 7, 8]
    ref_lp, ref_ent, big, log_s, _ = ref.forward(x[keep], np.minimum(t[keep], vocab - 1))
    assert np.abs(ent[keep] - ref_ent).max() < 2000 * R
    assert np.array_equal(st[keep, 0], big) and np.abs(st[keep, 1] - log_s).max() < 200 * R
    assert abs(lp[4] - ref_lp[0]) < (200 + 50) * R
    # gradients of the same rows
    import torch
    one = torch.ones(9, device="cuda")
    lp2, dx = gpu_lib.token_loss(X, _targets(t))
    db = gpu_lib.token_logprobs_backward(X, _targets(t), got.stats, dlogprob=-one)
    de = gpu_lib.token_logprobs_backward(X, _targets(t), got.stats, dlogprob=-one, dentropy=one,
                                         entropy=got.entropy)
    assert np.array_equal(np.isnan(_host(lp2)), np.isnan(lp))
    fin = np.isfinite(lp)
    assert np.array_equal(_host(lp2)[~fin & ~np.isnan(lp)], lp[~fin & ~np.isnan(lp)])
    assert np.abs(_host(lp2) - lp)[fin].max() < 400 * R * n
    for g in (dx, db, de):
        g = _host(g)
        assert (g[0] == 0).all()
        assert np.isnan(g[1]).all() and np.isnan(g[2]).all() and np.isnan(g[6]).all()
        assert np.isfinite(g[[3, 4, 5, 7, 8]]).all()
    for g in (dx, db):
        assert (_host(g)[8] == 0).all()
        assert abs(_host(g)[3].sum()) < 2 * (_half(dtype) + 300 * R)
        assert _host(g)[5, 3] == -1.0


def _check_gradient(got, x, t, dlp, de, dlse, dtype):
    want = ref.backward(x, t, dlp, de, dlse)
    _, ent, big, log_s, logp = ref.forward(x, t)
    fin = np.isfinite(logp)
    lp = np.where(fin, logp, 0.0)
    p = np.where(fin, np.exp(lp), 0.0)
    y = np.abs(lp + log_s[:, None])
    rel = (6 * y + 2 * np.abs(log_s[:, None]) + 190) * R
    coef = np.abs(dlse - np.where(t >= 0, dlp, 0))[:, None] + np.abs(de)[:, None] * (np.abs(lp) + ent[:, None])
    # the entropy given is the kernel's: 600 r of max(1, itself)
    own = np.abs(de)[:, None] * (2 * y + 600 * np.maximum(1, ent[:, None])) * R
    bound = (p + 2.0 ** -126) * (coef * (rel + 6 * R) + own) + 4 * R * np.abs(want) + 2.0 ** -126 * (1 + coef)
    at = np.maximum(t, 0)
    i = np.arange(len(t))
    bound[i, at] += 4 * R * np.abs(dlp)
    bound += (_half(dtype) + R) * np.abs(want)
    assert (np.abs(_host(got) - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_loss_and_backward(gpu_lib, vocab, dtype):
    import torch
    for rows in (1, 6) + ((700,) if vocab <= 1025 else ()):
        log(f"gradients {rows} x {vocab} {dtype}")
        x, t = _logits(vocab + rows, rows, vocab, masked=vocab // 5)
        t = np.where(np.isinf(x[np.arange(rows), np.maximum(t, 0)]), -1, t)
        X, T = _dev(x, dtype), _targets(t)
        x = _host(X)
        r = np.random.default_rng(9)
        a, b, c = r.standard_normal((3, rows)).astype(np.float32).astype(np.float64)
        v = lambda z: torch.from_numpy(z.astype(np.float32)).cuda()
        zero = np.zeros(rows)
        f = gpu_lib.token_logprobs(X, T)
        lp, dx = gpu_lib.token_loss(X, T, v(a))
        assert dx.dtype == X.dtype
        _check_gradient(dx, x, t, -a, zero, zero, dtype)
        want = ref.forward(x, t)
        assert (np.abs(_host(lp) - want[0]) <= (170 + 2 * np.abs(want[0]) + 6 * np.abs(want[3])) * R).all()
        lp1, dx1 = gpu_lib.token_loss(X, T)
        _check_gradient(dx1, x, t, -np.ones(rows), zero, zero, dtype)
        assert torch.equal(lp1, lp)
        bw = gpu_lib.token_logprobs_backward
        _check_gradient(bw(X, T, f.stats, dlogprob=v(a)), x, t, a, zero, zero, dtype)
        _check_gradient(bw(X, T, f.stats, dlogprob=v(a), dentropy=v(b), dlse=v(c), entropy=f.entropy),
                        x, t, a, b, c, dtype)
        _check_gradient(bw(X, None, f.stats, dlse=v(c)), x, t * 0 - 1, zero, zero, c, dtype)
        _check_gradient(bw(X, None, f.stats, dentropy=v(b), entropy=f.entropy), x, t * 0 - 1, zero, b,
                        zero, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [37, 3001, 20003, 140001])
def test_in_place_views_and_types(gpu_lib, vocab, dtype):
    """The gradient in place of the logits equals the one beside them; views of a wider buffer
    give the same and nothing beside them changes; results of the other type."""
    import torch
    log(f"in place {vocab} {dtype}")
    x, t = _logits(vocab, 5, vocab)
    X, T = _dev(x, dtype), _targets(t)
    w = torch.rand(5, device="cuda")
    f = gpu_lib.token_logprobs(X, T, top=9)
    _, dx = gpu_lib.token_loss(X, T, w)
    db = gpu_lib.token_logprobs_backward(X, T, f.stats, dlogprob=w, dentropy=w, entropy=f.entropy)
    ld = (vocab + 7) // 8 * 8 + 24
    wide = torch.full((7, ld), 5.0, dtype=X.dtype, device="cuda")
    view = wide[1:6, 16:16 + vocab]

    def same_outside():
        keep = wide.clone()
        keep[1:6, 16:16 + vocab] = 5.0
        assert (keep == 5.0).all()

    view.copy_(X)
    g = gpu_lib.token_logprobs(view, T, top=9)
    for p, q in zip(f, g):
        assert torch.equal(p, q)
    lp, out = gpu_lib.token_loss(view, T, w, out=view)
    assert out.data_ptr() == view.data_ptr() and torch.equal(view, dx)
    same_outside()
    view.copy_(X)
    gpu_lib.token_logprobs_backward(view, T, f.stats, dlogprob=w, dentropy=w, entropy=f.entropy, out=view)
    assert torch.equal(view, db)
    same_outside()
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    o = gpu_lib.empty_matrix(5, vocab, other, "cuda")
    gpu_lib.token_loss(X, T, w, out=o)
    assert torch.equal(o.to(X.dtype) if dtype == "bf16" else o, dx if dtype == "bf16" else dx.to(other))
    gpu_lib.token_logprobs_backward(X, T, f.stats, dlogprob=w, dentropy=w, entropy=f.entropy, out=o)
    assert torch.equal(o.to(X.dtype) if dtype == "bf16" else o, db if dtype == "bf16" else db.to(other))


def test_rows_without_a_target_may_hold_anything(gpu_lib):
    import torch
    log("rows without a target")
    x, _ = _logits(4, 6, 3000)
    X = _dev(x, "bf16")
    X[1], X[4] = float("nan"), float("inf")
    t = _targets([5, -1, 7, -100, -1, 9])
    lp, dx = gpu_lib.token_loss(X, t)
    f = gpu_lib.token_logprobs(X, t)
    db = gpu_lib.token_logprobs_backward(X, t, f.stats, dlogprob=-torch.ones(6, device="cuda"))
    for g in (dx, db):
        assert torch.isfinite(g).all() and (g[[1, 3, 4]] == 0).all() and g[[0, 2, 5]].any(dim=1).all()
    assert (lp[[1, 3, 4]] == 0).all() and (f.logprob[[1, 3, 4]] == 0).all()


@pytest.mark.parametrize("vocab", [5, 3000, 200003])
def test_rows_of_weight_zero_may_hold_anything(gpu_lib, vocab):
    """As for the backward call: no gradient, while the log probabilities are the rows' own."""
    import torch
    log(f"rows of weight zero {vocab}")
    x, _ = _logits(4, 5, vocab)
    X = _dev(x, "bf16")
    X[1], X[3] = float("nan"), float("inf")
    t, w = _targets([1, 2, 3, 4, 0]), torch.tensor([1.0, 0.0, 0.0, -0.0, 2.0], device="cuda")
    want = gpu_lib.token_logprobs(X, t)
    one = gpu_lib.token_loss(X[4:], t[4:], w[4:])
    lp, dx = gpu_lib.token_loss(X, t, w)
    assert torch.isfinite(dx).all() and (dx[1:4] == 0).all() and dx[[0, 4]].any(dim=1).all()
    assert torch.equal(dx[4:], one[1])
    assert torch.isnan(lp[[1, 3]]).all() and torch.isnan(want.logprob[[1, 3]]).all()
    # each within 170 + 2 |lp| + 6 log S (both below 20) steps of 2^-24 of the formula's
    assert (lp[[0, 2, 4]] - want.logprob[[0, 2, 4]]).abs().max() < 2 * 330 * R


def test_captured(gpu_lib):
    """Two graphs of calls and a larger eager call between their
    replays: every replay equals the eager results, new logits included."""
    import torch
    log("captured")
    x1, t1 = _logits(1, 2, 60000)
    x2, t2 = _logits(2, 3, 90000)
    x3, t3 = _logits(3, 9, 140000)
    A, B, C = _dev(x1, "bf16"), _dev(x2, "f32"), _dev(x3, "f32")
    T = [_targets(t) for t in (t1, t2, t3)]
    gpu_lib.token_logprobs(A, T[0], top=8)
    gpu_lib.token_loss(A, T[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for X, tt in ((A, T[0]), (B, T[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f = gpu_lib.token_logprobs(X, tt, top=8)
            d = gpu_lib.token_logprobs_backward(X, tt, f.stats, dlogprob=f.logprob, dentropy=f.entropy,
                                                entropy=f.entropy)
            outs.append((*f, d, *gpu_lib.token_loss(X, tt)))
        graphs.append(g)
    for k in range(3):
        A.mul_(0.9)
        B.add_(0.1)
        graphs[0].replay()
        gpu_lib.token_logprobs(C, T[2], top=32)
        graphs[1].replay()
        torch.cuda.synchronize()
        for (X, tt), o in zip(((A, T[0]), (B, T[1])), outs):
            f = gpu_lib.token_logprobs(X, tt, top=8)
            d = gpu_lib.token_logprobs_backward(X, tt, f.stats, dlogprob=f.logprob, dentropy=f.entropy,
                                                entropy=f.entropy)
            for p, q in zip(o, (*f, d, *gpu_lib.token_loss(X, tt))):
                assert torch.equal(p, q)


def test_two_streams(gpu_lib):
    """Calls on two streams at once."""
    import torch
    log("two streams")
    x1, t1 = _logits(1, 2, 100000)
    x2, t2 = _logits(2, 2, 100000)
    X = [_dev(x1, "bf16"), _dev(x2, "bf16")]
    T = [_targets(t1), _targets(t2)]
    want = [gpu_lib.token_logprobs(a, b, top=16) for a, b in zip(X, T)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for k in range(10):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                got[i].append(gpu_lib.token_logprobs(X[i], T[i], top=16))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for p, q in zip(g, want[i]):
                assert torch.equal(p, q)


def test_far_offsets(gpu_lib):
    """Rows whose offsets pass 2^32 elements."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GiB of free GPU memory are needed")
    log("far offsets")
    rows, ld = 66000, 1 << 17
    buf = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    v = buf[:, :72]
    x, t = _logits(6, rows, 72)
    X = _dev(x, "bf16", pad=0.0)
    v.copy_(X)
    T = _targets(t)
    f, g = gpu_lib.token_logprobs(X, T, top=3), gpu_lib.token_logprobs(v, T, top=3)
    for p, q in zip(f, g):
        assert torch.equal(p, q)
    _, dx = gpu_lib.token_loss(X, T)
    one = torch.ones(rows, device="cuda")
    db = gpu_lib.token_logprobs_backward(X, T, f.stats, dlogprob=one)
    gpu_lib.token_logprobs_backward(v, T, f.stats, dlogprob=one, out=v)
    assert torch.equal(v, db)
    v.copy_(X)
    gpu_lib.token_loss(v, T, out=v)
    assert torch.equal(v, dx)
    del buf, v
    torch.cuda.empty_cache()


def test_refusals(gpu_lib):
    import torch
    log("refusals")
    lib = gpu_lib
    X = torch.randn((4, 64), device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = lib.token_logprobs(X, t)
    z = torch.zeros(4, device="cuda")
    for call, error in (
            (lambda: lib.token_logprobs(X, t.int()), TypeError),
            (lambda: lib.token_logprobs(X, t[:3]), ValueError),
            (lambda: lib.token_logprobs(X, t.cpu()), ValueError),
            (lambda: lib.token_logprobs(X, t, top=-1), ValueError),
            (lambda: lib.token_logprobs(X, t, top=33), lib.MaoError),
            (lambda: lib.token_logprobs(X[:, :8], t, top=9), lib.MaoError),
            (lambda: lib.token_logprobs(X.half(), t), TypeError),
            (lambda: lib.token_logprobs(X.t(), t), ValueError),
            (lambda: lib.token_logprobs(X[0], t), ValueError),
            (lambda: lib.token_logprobs(X[:, :60].contiguous(), t), lib.MaoError),
            (lambda: lib.token_logprobs(X.clone().requires_grad_(True), t), RuntimeError),
            (lambda: lib.token_loss(X, t, z[:3]), ValueError),
            (lambda: lib.token_loss(X, t, z.bfloat16()), TypeError),
            (lambda: lib.token_loss(X, t, out=torch.empty((4, 56), device="cuda")), lib.MaoError),
            (lambda: lib.token_logprobs_backward(X, t, f.stats), lib.MaoError),
            (lambda: lib.token_logprobs_backward(X, t, f.stats[:3], dlogprob=z), ValueError),
            (lambda: lib.token_logprobs_backward(X, t, f.stats.double(), dlogprob=z), TypeError),
            (lambda: lib.token_logprobs_backward(X, None, f.stats, dlogprob=z), lib.MaoError),
            (lambda: lib.token_logprobs_backward(X, t, f.stats, dentropy=z), lib.MaoError),
            (lambda: lib.token_logprobs_backward(X, t, f.stats, dlse=z.double()), TypeError)):
        with pytest.raises(error):
            call()
    only = lib.token_logprobs(X, entropy=False)
    assert only.logprob is None and only.entropy is None and torch.equal(only.stats, f.stats)


@pytest.mark.parametrize("vocab", [5, 3000, 200003])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_targets_far_below_zero(gpu_lib, vocab, dtype):
    """A target below 0 is none whatever its lower 32 bits say: nothing of its row counts."""
    import torch
    log(f"targets far below zero {vocab} {dtype}")
    x, _ = _logits(4, 6, vocab)
    X = _dev(x, dtype)
    X[2] = float("nan")
    t = _targets([-(1 << 32) + 3, -(1 << 63) + 1, -(1 << 40), -(1 << 63), -(1 << 32) + 4, 2])
    f = gpu_lib.token_logprobs(X, t)
    assert (f.logprob[:5] == 0).all() and f.logprob[5] != 0
    one = torch.ones(6, device="cuda")
    for w in (None, one):
        lp, dx = gpu_lib.token_loss(X, t, w)
        assert (lp[:5] == 0).all() and (dx[:5] == 0).all() and lp[5] != 0 and dx[5].any()
    db = gpu_lib.token_logprobs_backward(X, t, f.stats, dlogprob=one)
    assert (db[:5] == 0).all() and db[5].any()


@pytest.mark.parametrize("vocab", [5, 3000, 200003])
def test_weight_zero_outside_the_vocabulary(gpu_lib, vocab):
    """A row of weight 0 gets zeros also where its target is outside the vocabulary."""
    import torch
    log(f"weight zero, target outside {vocab}")
    x, _ = _logits(4, 4, vocab)
    X = _dev(x, "bf16")
    t = _targets([vocab, 1, vocab + 7, vocab])
    lp, dx = gpu_lib.token_loss(X, t, torch.tensor([0.0, 1.0, -0.0, 1.0], device="cuda"))
    assert torch.isnan(lp[[0, 2, 3]]).all() and torch.isfinite(lp[1])
    assert (dx[[0, 2]] == 0).all() and torch.isnan(dx[3]).all()
    assert torch.isfinite(dx[1]).all() and dx[1].any()


@pytest.mark.parametrize("vocab", [5, 3000, 70000])
def test_backward_outside_the_vocabulary(gpu_lib, vocab):
    """A target outside the vocabulary makes NaN of its row through a gradient of its log
    probability alone: one that is 0 or not given, and the others' gradients, do not know it."""
    import torch
    log(f"backward, target outside {vocab}")
    x, _ = _logits(4, 3, vocab)
    X = _dev(x, "bf16")
    t, ok = _targets([vocab, 1, 2]), _targets([0, 1, 2])
    f = gpu_lib.token_logprobs(X, ok)
    one = torch.ones(3, device="cuda")
    bw = gpu_lib.token_logprobs_backward
    for kw in (dict(dlse=one), dict(dentropy=one, entropy=f.entropy)):
        assert torch.equal(bw(X, t, f.stats, **kw), bw(X, None, f.stats, **kw))
        zero = torch.tensor([0.0, 1.0, 1.0], device="cuda")
        assert torch.equal(bw(X, t, f.stats, dlogprob=zero, **kw), bw(X, ok, f.stats, dlogprob=zero, **kw))
    g = bw(X, t, f.stats, dlogprob=zero)
    assert (g[0] == 0).all() and torch.equal(g, bw(X, ok, f.stats, dlogprob=zero))
    g = bw(X, t, f.stats, dlogprob=one)
    assert torch.isnan(g[0]).all() and torch.isfinite(g[1:]).all()


@pytest.mark.parametrize("vocab", [5, 3000, 70000])
def test_equal_gradients_of_a_row_of_nan(gpu_lib, vocab):
    """Equal gradients of a row's log probability and of its log of the sum cancel in the
    probabilities' factor; a row with a NaN or +inf has NaN all the same, any other one the
    target's gradient alone."""
    import torch
    log(f"equal gradients {vocab}")
    x, _ = _logits(4, 4, vocab)
    X = _dev(x, "bf16")
    X[1, 2], X[3, 0] = float("nan"), float("inf")
    t = _targets([1, 2, 3, 4])
    f = gpu_lib.token_logprobs(X, t)
    two = torch.full((4,), 2.0, device="cuda")
    g = gpu_lib.token_logprobs_backward(X, t, f.stats, dlogprob=two, dlse=two)
    assert torch.isnan(g[[1, 3]]).all()
    want = torch.zeros_like(g)
    want[0, 1] = want[2, 3] = 2.0
    assert torch.equal(g[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_of_rows_read_twice(gpu_lib, dtype):
    """Rows beyond the registers, of both types: values against float64."""
    log(f"loss of long rows {dtype}")
    rows, vocab = 4, 200003
    x, t = _logits(8, rows, vocab, masked=vocab // 5)
    t = np.where(np.isinf(x[np.arange(rows), np.maximum(t, 0)]), -1, t)
    t[0] = int(np.argmax(x[0]))
    X, T = _dev(x, dtype), _targets(t)
    x = _host(X)
    import torch
    a = np.random.default_rng(9).standard_normal(rows).astype(np.float32).astype(np.float64)
    lp, dx = gpu_lib.token_loss(X, T, torch.from_numpy(a.astype(np.float32)).cuda())
    zero = np.zeros(rows)
    _check_gradient(dx, x, t, -a, zero, zero, dtype)
    want = ref.forward(x, t)
    assert (np.abs(_host(lp) - want[0]) <= (170 + 2 * np.abs(want[0]) + 6 * np.abs(want[3])) * R).all()


@pytest.mark.parametrize("vocab", [9000, 50304, 70000])
@pytest.mark.parametrize("offset", [256.0, -4096.0, 1e6])
def test_alternatives_of_rows_with_an_offset(gpu_lib, vocab, offset):
    """fp32 logits far from 0, no two alike but by chance: thousands share the upper 16 bits."""
    log(f"alternatives, offset {offset} {vocab}")
    x, t = _logits(vocab, 5, vocab)
    X = _dev(x + offset, "f32")
    got = gpu_lib.token_logprobs(X, _targets(t), top=20)
    assert np.array_equal(got.top_ids.cpu().numpy(), ref.top(_host(X), 20))
    want = np.take_along_axis(ref.forward(_host(X), t)[4], ref.top(_host(X), 20), axis=1)
    # y = x - M is exact here or off by r |y|, as always: the offset does not count
    assert (np.abs(_host(got.top_logprobs) - want) <= (400 + 4 * np.abs(want)) * R).all()
