"""The sums over a norm's row: as many roundings as a tree of the row's threads has levels."""
import numpy as np
import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("kind", ["residual", "inner"])
@pytest.mark.parametrize("D", [8192, 16384])
def test_parts_that_are_small_beside_another_are_not_lost_one_by_one(D, kind):
    """One square of 2^24 and 31 of 1, 256 channels apart, so in as many warps of a row: added to the large one in turn, each of
    them rounds away, and 31 U of the sum and 15.5 U of its root are gone.  In a tree the five levels over the warps can
    round once each (a thread's and a lane's other terms are 0): 5 U of the sum, 2.5 U of its root.  The mean and eps take 1 U
    more, the root itself two units in the last place, 4 U, and two products 2 U: 9.5 U."""
    x = torch.zeros(1, D, device="cuda")
    x[0, 0] = 2.0 ** 12
    x[0, 256:32 * 256:256] = 1.0
    w = torch.ones(D, device="cuda")
    off = []
    for eps in np.linspace(0.0, 40.0, 64, dtype=np.float32):
        if kind == "inner":
            y = sdm.gated_norm(x, w, eps=float(eps))
        else:
            y = sdm.residual_norm(x, weight=w, eps=float(eps))[0]
        want = 2.0 ** 12 / np.sqrt((2.0 ** 24 + 31) / D + float(eps))
        off.append(abs(y[0, 0].item() / want - 1) / U)
    assert max(off) <= 9.5, max(off)
