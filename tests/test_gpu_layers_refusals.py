"""What the layer calls refuse before anything is launched (GPU)."""
import pytest

from tests.helpers import log

pytestmark = pytest.mark.gpu


def _checkpoint(lib):
    import torch
    x = torch.randn((8, 72), device="cuda")
    return x, lib.q8_quantize(x)


def test_checkpoint_whose_parts_were_replaced(gpu_lib):
    """codes and scales are plain attributes: what Q8 refuses as it is made is also
    refused where it is used."""
    import torch
    log("replaced codes and scales")
    lib = gpu_lib
    x, _ = _checkpoint(lib)
    mean = torch.zeros(8, device="cuda")
    w = torch.randn((16, 72), device="cuda")
    dy = torch.randn((8, 16), device="cuda")

    def uses(q):
        yield lambda: lib.q8_dequantize(q)
        yield lambda: lib.q8_quantize(x, out=q)
        yield lambda: lib.layer_norm_backward(x, q, None, mean, mean)
        yield lambda: lib.linear_backward_input(dy, w, act="relu", preact=q)
        yield lambda: lib.linear_backward_weight(dy, q)

    def replaced(**parts):
        q = _checkpoint(lib)[1]
        for k, v in parts.items():
            setattr(q, k, v)
        return q

    _, q = _checkpoint(lib)
    wide = torch.zeros((8, 256), dtype=torch.int8, device="cuda")
    for bad, error in ((replaced(scales=q.scales[:3]), ValueError),
                       (replaced(scales=q.scales[:, :2]), ValueError),
                       (replaced(scales=q.scales[0]), ValueError),
                       (replaced(scales=torch.zeros((8, 8), dtype=torch.uint8, device="cuda")[:, ::2]),
                        ValueError),
                       (replaced(scales=q.scales.to(torch.int8)), TypeError),
                       (replaced(codes=wide[:, ::3][:, :72]), ValueError),
                       (replaced(codes=q.codes.float()), TypeError),
                       (replaced(codes=q.codes.view(torch.uint8)), TypeError),
                       (replaced(scales=q.scales.cpu()), ValueError)):
        for use in uses(bad):
            with pytest.raises(error):
                use()


def test_quantise_into_something_else(gpu_lib):
    import types

    import torch
    log("quantise into something else")
    x, q = _checkpoint(gpu_lib)
    with pytest.raises(TypeError):
        gpu_lib.q8_quantize(x, out=types.SimpleNamespace(codes=torch.zeros((8, 96), device="cuda")[:, :72],
                                                         scales=q.scales))


def test_tensors_that_autograd_follows(gpu_lib):
    """The calls record no graph: with gradients on, a tensor that requires one is
    refused rather than cut off; with gradients off it is an ordinary tensor."""
    import torch
    log("requires_grad")
    lib = gpu_lib
    x, w, b = (torch.randn(s, device="cuda") for s in ((8, 72), (16, 72), (16,)))
    dy, z, g = (torch.randn(s, device="cuda") for s in ((8, 16), (8, 72), (72,)))
    _, mean, rstd = lib.layer_norm(x, g)
    q = lib.q8_quantize(x)
    r = lambda t: t.clone().requires_grad_(True)
    calls = [(lib.linear, (x, w, b), {}), (lib.layer_norm, (x, g, g), {}),
             (lib.q8_quantize, (x,), {}), (lib.layer_norm_backward, (x, z, g, mean, rstd), {}),
             (lib.layer_norm_backward, (x, q, g, mean, rstd), {}),
             (lib.linear_backward_input, (dy, w), {"act": "silu", "preact": z}),
             (lib.linear_backward_weight, (dy, x), {})]
    for fn, args, kw in calls:
        for i, a in enumerate(args):
            if a is q:
                continue
            some = [*args[:i], torch.nn.Parameter(a) if i % 2 else r(a), *args[i + 1:]]
            with pytest.raises(RuntimeError, match="no_grad"):
                fn(*some, **kw)
            with torch.no_grad():
                fn(*some, **kw)
            with torch.inference_mode():
                fn(*some, **kw)
        fn(*args, **kw)
    with pytest.raises(RuntimeError, match="no_grad"):
        lib.linear_backward_input(dy, w, act="silu", preact=r(z))
    with pytest.raises(RuntimeError, match="no_grad"):
        lib.linear(x, w, residual=r(dy))


def test_vector_gradients_that_are_not_wanted(gpu_lib):
    """False leaves a vector gradient out: the rest comes out bit for bit the same, and
    the C entry point asks for no workspace for it."""
    import ctypes

    import torch
    log("unwanted vector gradients")
    lib = gpu_lib
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x, dy = (torch.randn((300, 72), generator=gen, device="cuda") for _ in range(2))
    gamma = torch.rand(72, generator=gen, device="cuda")
    _, mean, rstd = lib.layer_norm(x, gamma)
    dx, dg, db = lib.layer_norm_backward(dy, x, gamma, mean, rstd)
    for wg, wb in ((False, None), (None, False), (False, False)):
        got = lib.layer_norm_backward(dy, x, gamma, mean, rstd, dgamma=wg, dbeta=wb)
        assert torch.equal(got[0], dx)
        assert got[1] is None if wg is False else torch.equal(got[1], dg)
        assert got[2] is None if wb is False else torch.equal(got[2], db)
    for rows, n in ((300, 72), (5000, 40)):  # the second with K split
        x = torch.randn((rows, 56), generator=gen, device="cuda").bfloat16()
        dy = torch.randn((rows, n), generator=gen, device="cuda").bfloat16()
        for act in ("none", "gelu"):
            dw, db = lib.linear_backward_weight(dy, x, x_act=act)
            got, none = lib.linear_backward_weight(dy, x, x_act=act, dbias=False)
            assert none is None and torch.equal(got, dw)
            twice, none = lib.linear_backward_weight(dy, x, x_act=act, out=got, dbias=False,
                                                     accumulate=True)
            full = dw.clone()
            lib.linear_backward_weight(dy, x, x_act=act, out=full, dbias=db, accumulate=True)
            assert none is None and torch.equal(twice, full)
    # 8 rows: one part, nothing rebuilt; without dbias no workspace at all
    x, dy = (torch.randn((8, 72), generator=gen, device="cuda") for _ in range(2))
    want, _ = lib.linear_backward_weight(dy, x)
    out = torch.empty_like(want)
    c = lib.load()
    call = lambda db: c.mao_linear_backward_weight(
        lib.mat(dy), ctypes.byref(lib.mat(x)), None, 0, lib.mat(out), db, 0, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert c.mao_linear_backward_weight_workspace_size(8, 72, 72, lib.F32, 0) > 0
    assert call(torch.empty(72, device="cuda").data_ptr()) == 7  # MAO_E_WORKSPACE
    assert call(None) == 0
    assert torch.equal(out, want)


def test_results_that_do_not_fit_memory(gpu_lib):
    """torch's own error, which programs catch; the next call is unharmed."""
    import torch
    log("out of memory")
    lib = gpu_lib
    x = torch.randn((1 << 20, 8), device="cuda").bfloat16()
    with pytest.raises(torch.OutOfMemoryError):
        lib.linear(x, x)  # 2^40 results
    y = lib.linear(x[:40], x[:24])
    want = x[:40].double() @ x[:24].double().t().contiguous()
    assert float((y.double() - want).abs().max()) < 0.1
