"""The backward norms' workgroups over more than one row each, in every launch
shape, read by 16 bytes and by element; formulas and tolerances as in
test_gpu_block_norm.py.  And what a row's bits depend on."""

import pytest
import torch

from test_gpu_block_norm import BF16, EPS, F32, args, check_backward, check_forward, make

pytestmark = pytest.mark.gpu


# twice the workgroups of the launch at least, on a GPU of 256 CUs
@pytest.mark.parametrize("T,H", [(9000, 40), (9000, 33), (1100, 1024), (1100, 1001), (1100, 4096), (1100, 2049),
                                 (600, 5000), (600, 5001), (600, 12288), (600, 9001)])
@pytest.mark.parametrize("x,y,gate", [(BF16, BF16, "channel"), (BF16, F32, "token"), (F32, F32, "channel"),
                                      (BF16, BF16, "full"), (BF16, None, "none"), (F32, None, "none")])
def test_several_rows_a_workgroup(lib, T, H, x, y, gate):
    check_backward(lib, make(T, H, x, y, gate, post=y is not None, seed=T + H))


@pytest.mark.parametrize("H", [520, 2048, 7168])
def test_bits_at_another_stride(lib, H):
    """Strides of whole 16 bytes, and any batch on one side of the number of CUs
    (which counts for rows of 4097 to 8192)."""
    c = make(65, H, BF16, BF16, "channel", seed=23)
    out, n = check_forward(lib, c)
    wide = {k: torch.zeros((65, H + 24), dtype=BF16, device="cuda") for k in ("x", "y")}
    for k in wide:
        wide[k][:, :H] = c[k]
    for T in (65, 1, 20):
        o2, n2 = lib.block_norm(wide["x"][:T, :H], wide["y"][:T, :H], res_scale=0.875, eps=EPS, **args(c))
        assert torch.equal(o2, out[:T]) and torch.equal(n2, n[:T])
