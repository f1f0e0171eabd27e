"""The fp64 oracle of the log-probabilities' gradient, from the logits alone,
against torch's automatic differentiation in fp64 (CPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ends_ref as R


@pytest.mark.parametrize("scale", [1.0, 0.7, 1e4])
@pytest.mark.parametrize("offset", [0.0, 1e3, -1e5])
def test_gradient(scale, offset):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((9, 13)) * 3 / scale + offset
    x[4, 3:9] = -np.inf
    x[5] = -1e9
    t = np.array([0, 12, -100, 13, 1, 2, 3, 5, 6])
    up = rng.standard_normal(9)
    up[7] = 0.0
    live = [0, 1, 4, 5, 6, 7, 8]
    lx = torch.tensor(x, requires_grad=True)
    ls = torch.log_softmax(lx[live] * scale, 1)
    (want,) = torch.autograd.grad((ls[range(7), t[live]] * torch.tensor(up[live])).sum(), [lx])
    got = R.token_logp_gradient(x, t, scale, up)
    # z itself is rounded to 2^-53 of the offset
    np.testing.assert_allclose(got, torch.nan_to_num(want), rtol=1e-11 + 1e-15 * abs(offset) * scale, atol=1e-13)
    assert not got[2].any() and not got[3].any() and not got[7].any()
    assert np.abs(got.sum(1)).max() < 1e-11 * scale
    assert not R.token_logp_gradient(np.full((1, 4), -np.inf), np.array([1]), scale, np.ones(1)).any()
