"""The join's kernels past their first round of rows, in every form (GPU).

A workgroup goes on to a next row group only where the rows are more than the workgroups of one grid
hold: 256 CUs' 2048 threads forward, 256 workgroups of at most 1024 threads backward. Each
case here has two full rounds of its form and three rows more.
"""
import numpy as np
import pytest

from tests.helpers import log
from tests.test_gpu_residual_norm import Case, _check_forward, _run, _vec

pytestmark = pytest.mark.gpu

# columns near a form's limit: rows of a round, forward with a bf16 stream and block and with fp32 in
# one of them, backward the same
FORMS = {253: (8192, 8192, 4096, 4096), 509: (8192, 4096, 4096, 2048), 765: (8192, 2048, 1280, 1280),
         1021: (4096, 2048, 2048, 1024), 1533: (4096, 1024, 1280, 512), 2045: (2048, 1024, 1024, 512),
         2557: (1536, 512, 768, 256), 4093: (1024, 512, 512, 256), 6141: (1024, 512, 256, 256),
         8189: (512, 512, 256, 256), 16381: (512, 512, 256, 256)}
TYPES = [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")]


class Rows:
    """Some rows of a case, as _check_forward takes them."""

    def __init__(self, c, x, b, gates, idx):
        self.X, self.B = x[idx], b[idx]
        self.g = gates[idx].double().cpu().numpy() if gates is not None else c["g"]
        self.n1, self.n2, self.post, self.pre = c["n1"], c["n2"], c["n1"][0], c["n2"][0]
        self.xs, self.bs, self.xt, self.bt = c["xs"], c["bs"], c["xt"], c["bt"]


def _rows_of(seed, rows, cols, dtype):
    """Rows of changing size, some of zeros, in a buffer whose padding holds NaN."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((rows, (cols + 7) // 8 * 8), float("nan"), device="cuda",
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x = x * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda")) + 0.3
    x[1 + seed::7] = 0.0
    buf[:, :cols] = x
    return buf[:, :cols]


@pytest.mark.parametrize("cols", FORMS)
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate", ["vector", "matrix"])
def test_forward(gpu_lib, cols, types, gate):
    """Rows around the ends of the rounds and a sample of all against float64; every row
    bit for bit what calls of less than a round give."""
    import torch
    xt, bt = types
    each = FORMS[cols][0 if xt == bt == "bf16" else 1]
    rows = 2 * each + 3
    log(f"forward rounds {rows} x {cols} {types} {gate}")
    r = np.random.default_rng(cols)
    x, b = _rows_of(1, rows, cols, xt), _rows_of(2, rows, cols, bt)
    post, pre = ("layer", "rms") if gate == "vector" else ("rms", "layer")
    kw = dict(post=post, pre=pre, post_gamma=_vec(1 + 0.3 * r.standard_normal(cols)),
              pre_gamma=_vec(1 + 0.3 * r.standard_normal(cols)), x_scale=0.75, b_scale=-1.5)
    kw["post_beta" if post == "layer" else "pre_beta"] = _vec(0.2 * r.standard_normal(cols))
    gates = _rows_of(3, rows, cols, bt) if gate == "matrix" else None
    vec = None if gates is not None else _vec(0.5 + 0.5 * r.standard_normal(cols))
    host = lambda k: kw[k].double().cpu().numpy() if k in kw else 0.0  # noqa: E731
    c = dict(n1=(post, host("post_gamma"), host("post_beta")), xs=0.75, bs=-1.5, xt=xt, bt=bt,
             n2=(pre, host("pre_gamma"), host("pre_beta")),
             g=None if vec is None else vec.double().cpu().numpy())
    got = gpu_lib.residual_norm(x, b, gate=vec if gates is None else gates, **kw)
    ends = [e + d for e in (0, each, 2 * each) for d in (-2, -1, 0, 1, 2)]
    idx = sorted({e for e in ends if 0 <= e < rows} | set(r.integers(0, rows, 60).tolist()))
    _check_forward(Rows(c, x, b, gates, idx), [t[idx] for t in got])
    for lo in range(0, rows, each - 1):
        part = slice(lo, min(rows, lo + each - 1))
        one = gpu_lib.residual_norm(x[part], b[part], gate=vec if gates is None else gates[part], **kw)
        for p, q in zip(got, one):
            assert torch.equal(p[part], q)


# (wider rows of all types go through several rounds in test_wide_rows_in_turn)
@pytest.mark.parametrize("cols", [c for c in FORMS if c <= 4093])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_both_directions(gpu_lib, cols, types):
    """Gradients and their column sums, after several rounds, against float64."""
    rows = 2 * FORMS[cols][2 if types == ("bf16", "bf16") else 3] + 3
    log(f"backward rounds {rows} x {cols} {types}")
    _run(gpu_lib, Case(cols, rows, cols, *types, "layer", "layer", "vector"))
