"""moe_w4_linear where the parts of K that its wavefronts take end unevenly: the
routed form whose experts get few entries (parts of 1024 inputs), with tails of
one to seven halves, several passes over one expert's entries, and either
scale type and zero points; dense products' bits over every number of x rows.
Tolerances as in test_gpu_w4.py."""

import pytest
import torch

from test_gpu_w4 import BF16, F32, check, make

pytestmark = pytest.mark.gpu

# T, E, k with 3 T k <= 8 E: every expert has entries to look for, or only the touched ones
FEW = [(10, 16, 4), (3, 64, 4)]
PARTS = [(160, 32), (768, 32), (768, 64), (768, 128), (1152, 32), (1152, 64), (1152, 128), (1536, 64),
         (1536, 256), (1536, 512), (2080, 32), (9344, 128), (10240, 2048)]


@pytest.mark.parametrize("T,E,k", FEW)
@pytest.mark.parametrize("K,G", PARTS)
@pytest.mark.parametrize("scale,zero", [(BF16, True), (BF16, False), (F32, True), (F32, False)])
def test_routed_parts(lib, T, E, k, K, G, scale, zero):
    assert 3 * T * k <= 8 * E
    N = 36 if K < 9000 else 18
    check(lib, make(T, N, K, G, scale, zero, E, k, seed=K + G))
    check(lib, make(T, N, K, G, scale, zero, E, k, seed=K + G + 1), swiglu=True)
    check(lib, make(T, N, K, G, scale, zero, E, k, slots=True, weights=True, seed=K + G + 2), y_dtype="bf16")


@pytest.mark.parametrize("T,E", [(32, 128), (40, 16)])
@pytest.mark.parametrize("K,G", [(256, 64), (1152, 128), (2304, 32)])
def test_one_expert_takes_several_passes(lib, T, E, K, G):
    """One expert's entries in sets of eight, one pass after the other."""
    c = make(T, 40, K, G, BF16, True, E, 1, seed=T + K)
    c["ids"].fill_(E - 3)
    check(lib, c)
    check(lib, c, swiglu=True)


@pytest.mark.parametrize("K,G", [(1024, 128), (1120, 32), (2496, 64)])
def test_same_bits_for_any_number_of_rows(lib, K, G):
    """One, two and four sets of eight rows, and two rows of the grid."""
    c = make(70, 100, K, G, seed=K)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    rows = torch.cat([lib.w4_linear(W, c["x"][t:t + 1]) for t in range(70)])
    for T in (5, 12, 20, 32, 33, 70):
        assert torch.equal(lib.w4_linear(W, c["x"][:T]), rows[:T]), T
