"""The Python side of the layer operators on the host: refusals that need no GPU."""
import pytest

import matrix_aware_optimizers_amd as mao


@pytest.mark.parametrize("name", ["float16", "float64", "int8", "float8_e4m3fn"])
def test_unsupported_result_types_are_refused(name):
    """... and not replaced by a supported one. (CPU tensors: refused in any case, but
    with another error.)"""
    torch = pytest.importorskip("torch")
    dtype = getattr(torch, name)
    x = torch.zeros((4, 32))
    q = mao.Q8(torch.zeros((4, 32), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.uint8))
    with pytest.raises(TypeError):
        mao.q8_dequantize(q, dtype=dtype)
    with pytest.raises(TypeError):
        mao.linear_backward_weight(x, x, dtype=dtype)


def test_unknown_names_are_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 32))
    with pytest.raises(ValueError):
        mao.linear(x, x, act="swish")
