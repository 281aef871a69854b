"""Layer operators on matrices whose offsets pass 32 bits (GPU).

Views of few columns and a very long leading dimension: offsets reach beyond 2^32
elements while the work stays small. Every call must equal the same call on compact
copies bit for bit.
"""
import pytest

from tests.helpers import log

pytestmark = pytest.mark.gpu

ROWS, LD = 70001, 65536  # 70001 * 65536 > 2^32


def _far(t, buf):
    """t's values in a view of buf (rows x LD)."""
    v = buf[:t.shape[0], :t.shape[1]]
    v.copy_(t)
    return v


@pytest.fixture(scope="module")
def buffers():
    import torch
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GiB of free GPU memory are needed")
    bufs = [torch.empty((ROWS, LD), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    yield bufs
    del bufs
    torch.cuda.empty_cache()


def _randn(seed, *shape):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _same(a, b):
    import torch
    a = a if isinstance(a, (list, tuple)) else [a]
    b = b if isinstance(b, (list, tuple)) else [b]
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_layer_norm_far(gpu_lib, buffers):
    import torch
    log("layer norm, far offsets")
    x, dy, gam = _randn(1, ROWS, 72), _randn(2, ROWS, 72), torch.rand(72, device="cuda") + 0.5
    want = gpu_lib.layer_norm(x, gam, None)
    fx, fdy = _far(x, buffers[0]), _far(dy, buffers[1])
    out = buffers[2][:, :72]
    got = gpu_lib.layer_norm(fx, gam, None, out=out)
    assert got[0].data_ptr() == out.data_ptr()
    _same(got, want)
    _same(gpu_lib.layer_norm_backward(fdy, fx, gam, want[1], want[2], add=fdy),
          gpu_lib.layer_norm_backward(dy, x, gam, want[1], want[2], add=dy))


def test_linear_far(gpu_lib, buffers):
    log("linear, far offsets")
    x, w, res = _randn(3, ROWS, 72), _randn(4, 40, 72), _randn(5, ROWS, 40)
    fx, fres, out = _far(x, buffers[0]), _far(res, buffers[1]), buffers[2][:, :40]
    want = gpu_lib.linear(x, w, act="silu", residual=res)
    _same(gpu_lib.linear(fx, w, act="silu", residual=fres, out=out), want)
    # a weight with far rows: the forward product of a token, and of a batch
    big_w, t = _randn(6, ROWS, 72), x[:3]
    fw = _far(big_w, buffers[0])
    _same(gpu_lib.linear(t, fw), gpu_lib.linear(t, big_w))
    _same(gpu_lib.linear(x[:100], fw), gpu_lib.linear(x[:100], big_w))


def test_linear_gradients_far(gpu_lib, buffers):
    log("linear gradients, far offsets")
    dy, w, z = _randn(7, ROWS, 40), _randn(8, 40, 72), _randn(9, ROWS, 72)
    fdy, fz = _far(dy, buffers[0]), _far(z, buffers[1])
    _same(gpu_lib.linear_backward_input(fdy, w, act="gelu", preact=fz, out=buffers[2][:, :72]),
          gpu_lib.linear_backward_input(dy, w, act="gelu", preact=z))
    for act in ("none", "relu"):
        _same(gpu_lib.linear_backward_weight(fdy, fz, x_act=act),
              gpu_lib.linear_backward_weight(dy, z, x_act=act))


def test_checkpoint_far(gpu_lib, buffers):
    import torch
    log("checkpoints, far offsets")
    x = _randn(10, ROWS, 72)
    fx = _far(x, buffers[0])
    near = gpu_lib.q8_quantize(x, "int8")
    codes = buffers[1].view(torch.int8)[:, :72]  # ROWS x 72, rows 2 LD apart
    scales = torch.empty((ROWS, 3), dtype=torch.uint8, device="cuda")
    far = gpu_lib.q8_quantize(fx, out=gpu_lib.Q8(codes, scales))
    _same([far.codes, far.scales], [near.codes, near.scales])
    _same(gpu_lib.q8_dequantize(far, out=buffers[2][:, :72]), gpu_lib.q8_dequantize(near))
    dy, w = _randn(11, ROWS, 40), _randn(12, 40, 72)
    _same(gpu_lib.linear_backward_input(dy, w, act="silu", preact=far),
          gpu_lib.linear_backward_input(dy, w, act="silu", preact=near))
    _same(gpu_lib.linear_backward_weight(dy, far), gpu_lib.linear_backward_weight(dy, near))
