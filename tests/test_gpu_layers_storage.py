"""Layer operators on tensors whose storage ends with their last element (GPU).

An fp32 run of 8 columns is two 16-byte pieces; where a row ends within the first,
the second may lie past the allocation and must not be read. Every call must equal
the same call on padded copies bit for bit.
"""
import pytest

from tests.helpers import log

pytestmark = pytest.mark.gpu


def _end_of_flat(rows, cols, values):
    """One row of 4 k columns: the last elements of a flat buffer of 2 MiB (a whole
    mapping of the allocator)."""
    import torch
    flat = torch.zeros(1 << 19, device="cuda")
    v = flat[-cols:].view(1, cols)
    v.copy_(values)
    return v


def _right_half(rows, cols, values):
    """The last columns of a buffer whose rows are whole."""
    import torch
    ld = (cols + 7) // 8 * 8
    buf = torch.zeros((rows, ld), device="cuda")
    v = buf[:, ld - cols:]
    v.copy_(values)
    return v


def _last_row(rows, cols, values):
    """A contiguous matrix's last row."""
    import torch
    buf = torch.zeros((4, cols), device="cuda")
    v = buf[3:]
    v.copy_(values)
    return v


VIEWS = [(_end_of_flat, 1, 4), (_end_of_flat, 1, 36), (_right_half, 5, 4), (_right_half, 40, 12),
         (_right_half, 130, 516), (_last_row, 1, 12), (_last_row, 1, 4), (_last_row, 1, 44)]


def _same(a, b):
    import torch
    a = a if isinstance(a, (list, tuple)) else [a]
    b = b if isinstance(b, (list, tuple)) else [b]
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def _padded(t):
    import torch
    buf = torch.zeros((t.shape[0], (t.shape[1] + 15) // 8 * 8), device="cuda")
    v = buf[:, :t.shape[1]]
    v.copy_(t)
    return v


@pytest.mark.parametrize("make,rows,cols", VIEWS)
def test_rows_that_end_with_their_storage(gpu_lib, make, rows, cols):
    import torch
    log(f"storage ends with the row: {make.__name__} {rows} x {cols}")
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)

    def new():
        t = make(rows, cols, torch.randn((rows, cols), generator=g, device="cuda"))
        assert t.data_ptr() % 16 == 0
        return t

    lib = gpu_lib
    x, dy, add = new(), new(), new()
    px, pdy, padd = _padded(x), _padded(dy), _padded(add)
    gamma = torch.rand(cols, generator=g, device="cuda") + 0.5
    y, mean, rstd = lib.layer_norm(px, gamma, None)
    _same(lib.layer_norm(x, gamma, None, out=new()), [y, mean, rstd])
    _same(lib.layer_norm_backward(dy, x, gamma, mean, rstd, add=add, out=new()),
          lib.layer_norm_backward(pdy, px, gamma, mean, rstd, add=padd))
    # the joining gradient in another type than dY's
    bdy = lib.padded(pdy.bfloat16())
    _same(lib.layer_norm_backward(bdy, x, gamma, mean, rstd, add=add),
          lib.layer_norm_backward(bdy, px, gamma, mean, rstd, add=padd))
    for fmt in ("int8", "e4m3"):
        a, b = lib.q8_quantize(x, fmt), lib.q8_quantize(px, fmt)
        _same([a.codes.view(torch.int8), a.scales], [b.codes.view(torch.int8), b.scales])
        _same(lib.q8_dequantize(a, out=new()), lib.q8_dequantize(b, dtype=torch.float32))
    # as every operand of the products (few and many rows, short and split K)
    for k in (24, 1608):
        w = lib.padded(torch.randn((cols, k), generator=g, device="cuda"))
        h = lib.padded(torch.randn((rows, k), generator=g, device="cuda"))
        z, pz = new(), _padded(px)
        _same(lib.linear(h, w, act="silu", residual=add, preact=z, out=new()),
              lib.linear(h, w, act="silu", residual=padd, preact=pz))
        _same(z, pz)
        wt = lib.padded(torch.randn((k, cols), generator=g, device="cuda"))
        _same(lib.linear(x, wt), lib.linear(px, wt))
        _same(lib.linear_backward_input(h, wt, act="gelu", preact=x, add=add, out=new()),
              lib.linear_backward_input(h, wt, act="gelu", preact=px, add=padd))
        _same(lib.linear_backward_input(dy, w), lib.linear_backward_input(pdy, w))
        for act in ("none", "silu"):
            _same(lib.linear_backward_weight(h, x, x_act=act),
                  lib.linear_backward_weight(h, px, x_act=act))
        _same(lib.linear_backward_weight(dy, h), lib.linear_backward_weight(pdy, h))
        # the results' own storage: dW has as many rows as h has columns
        out = _right_half(k, cols, torch.ones((k, cols), device="cuda"))
        pout, db, pdb = _padded(out), torch.zeros(k, device="cuda"), torch.zeros(k, device="cuda")
        _same(lib.linear_backward_weight(h, x, out=out, dbias=db, accumulate=True),
              lib.linear_backward_weight(h, px, out=pout, dbias=pdb, accumulate=True))


def test_bf16_products_with_fp32_ends(gpu_lib):
    """fp32 residual, pre-activation and result of bf16 operands."""
    import torch
    log("storage ends with the row: bf16 operands, fp32 results")
    lib = gpu_lib
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for rows, k, n in ((70, 48, 12), (200, 1600, 132), (2051, 776, 3076)):
        x = torch.randn((rows, k), generator=g, device="cuda").bfloat16()
        w = torch.randn((n, k), generator=g, device="cuda").bfloat16()
        wt = lib.padded(w.t().contiguous())
        v = torch.randn((rows, n), generator=g, device="cuda")
        res = _right_half(rows, n, v)
        _same(lib.linear(x, w, act="gelu", residual=res, out=_right_half(rows, n, v)),
              lib.linear(x, w, act="gelu", residual=_padded(v), out=_padded(v)))
        _same(lib.linear_backward_input(x, wt, act="gelu", preact=res, add=res),
              lib.linear_backward_input(x, wt, act="gelu", preact=_padded(v), add=_padded(v)))
