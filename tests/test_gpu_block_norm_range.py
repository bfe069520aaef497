"""moe_block_norm and its backward pass on rows far from 1, against the
formulas in float64, at the tolerances of test_gpu_block_norm.py: relative to
the magnitudes that enter a value, so the rows' scale does not change them."""

import pytest
import torch

from test_gpu_block_norm import BF16, C_ROW, EPS, F32, args, close, gradients, make, reference

pytestmark = pytest.mark.gpu


def scaled(c, name, scale):
    c[name] = (c[name].float() * scale).to(c[name].dtype)
    return c


def check_forward(lib, c, eps):
    out, n = lib.block_norm(c["x"], c["y"], res_scale=0.875, eps=eps, **args(c))
    want_out, mag_out, want_n, mag_n = reference(c, 0.875, eps)
    if out is not None:
        close(out, want_out, mag_out, C_ROW, "out")
    if n is not None:
        close(n, want_n, mag_n, C_ROW, "n")


def check_backward(lib, c, eps):
    got = lib.block_norm_backward(c["grad_out"], c["grad_n"], c["x"], c["y"], res_scale=0.875, eps=eps, **args(c))
    want, mag = gradients(c, 0.875, eps)
    for k in want:
        # column sums add at most one rounding a token and 80 over the workgroups
        close(got[k], want[k], mag[k], 2 * C_ROW + (c["x"].shape[0] + 80 if got[k].dim() == 1 else 0), k)


@pytest.mark.parametrize("T,H", [(3, 200), (2, 1001), (4, 4096), (2, 8192), (2, 9000)])
@pytest.mark.parametrize("scale,eps", [(1e15, EPS), (3e12, EPS), (1e-14, 0.0), (1e-12, 0.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_loud_and_quiet_rows(lib, T, H, scale, eps, dtype):
    """The gradient is about 1/rms, whose cube would leave float32.  The stored
    stream and the block's output are taken one at a time, so that the term in
    question is not lost beside a larger one."""
    c = scaled(make(T, H, dtype, None, seed=17), "x", scale)
    c["grad_out"] = None
    check_backward(lib, c, eps)
    for gate in ("channel", "token"):
        check_backward(lib, scaled(make(T, H, dtype, dtype, gate, nxt=False, seed=18), "y", scale), eps)


@pytest.mark.parametrize("T,H", [(3, 200), (2, 1001), (4, 4096), (300, 7168), (2, 9000), (2, 16384)])
@pytest.mark.parametrize("scale,eps", [(1.2e19, EPS), (1e18, EPS), (4e-15, 0.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_up_to_the_largest_mean_square(lib, T, H, scale, eps, dtype):
    """A mean square of 1.4e38 is finite in float32, the row's sum of squares
    and the largest squares are not; and 2^-100 at the other end."""
    c = scaled(make(T, H, dtype, None, seed=19), "x", scale)
    c["grad_out"] = None
    check_forward(lib, c, eps)
    check_backward(lib, c, eps)
    for gate in ("channel", "token"):
        c = scaled(make(T, H, dtype, dtype, gate, nxt=False, seed=20), "y", scale)
        check_forward(lib, c, eps)
        check_backward(lib, c, eps)
    # a quiet block joins a quiet stream: out and its norm at that scale
    c = scaled(make(T, H, dtype, F32, post=False, seed=21), "x", scale)
    check_forward(lib, scaled(c, "y", scale), eps)


@pytest.mark.parametrize("H", [136, 1001, 2048, 8192])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_block_without_its_norm(lib, H, gate, dtype):
    """Without w_post and w_next the gradient of y is gate * grad_out whatever y is."""
    c = make(5, H, dtype, dtype, gate, post=False, nxt=False, seed=22)
    clean = lib.block_norm_backward(c["grad_out"], None, c["x"], c["y"], res_scale=0.875, eps=EPS, **args(c))
    c["y"][1, 5], c["y"][3, 7] = float("inf"), float("nan")
    got = lib.block_norm_backward(c["grad_out"], None, c["x"], c["y"], res_scale=0.875, eps=EPS, **args(c))
    assert torch.equal(got["y"], clean["y"]) and torch.equal(got["x"], clean["x"])
