"""Numbers of groups that do not fit an int are refused, not cut to one that does."""
import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [2 ** 32 + 1, 2 ** 32 + 4, 2 ** 40, -1, 0, 2 ** 70])
def test_groups_that_are_no_number_of_groups(groups):
    x, w = torch.randn(3, 64, device="cuda"), torch.ones(64, device="cuda")
    for call in (lambda: sdm.gated_norm(x, w, groups=groups), lambda: sdm.gated_norm_backward(x, w, x, groups=groups),
                 lambda: sdm.residual_norm(x, x.clone(), after=w, groups=groups),
                 lambda: sdm.gated_norm(x[:, :0], w[:0], groups=groups)):
        with pytest.raises((ValueError, OverflowError)):
            call()
