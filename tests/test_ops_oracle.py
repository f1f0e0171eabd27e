"""Pins of the fp64 oracle of the training operators (CPU): published answers
of the generator, and every gradient against central differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import ops_ref as R


@pytest.mark.parametrize("word,key,want", [
    (0, 0, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (0xFFFFFFFF, 0xFFFFFFFF, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
])
def test_philox_known_answers(word, key, want):
    got = R.philox([word] * 4, [key] * 2)
    assert tuple(int(v) for v in got) == want


def test_philox_known_answer_of_pi_digits():
    got = R.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0])
    assert tuple(int(v) for v in got) == (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_mask_rate_and_independence():
    a = R.keep_mask(200, 1001, 0.25, 7, 3)
    # 200200 draws: 5 standard deviations of the kept share are 0.0048
    assert abs(a.mean() - 0.75) < 0.005
    for other in (R.keep_mask(200, 1001, 0.25, 8, 3), R.keep_mask(200, 1001, 0.25, 7, 4),
                  R.keep_mask(200, 1001, 0.25, 7 + (1 << 40), 3)):
        # independent masks agree with probability 0.75^2 + 0.25^2
        assert abs((a == other).mean() - 0.625) < 0.006
    assert np.array_equal(a[50:60], R.keep_mask(10, 1001, 0.25, 7, 3, first_row=50))
    assert R.keep_mask(5, 9, 0.0, 1, 1).all() and not R.keep_mask(5, 9, 1.0, 1, 1).any()


def _difference(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_gradients_against_differences(affine):
    rng = np.random.default_rng(3)
    x, dy, v = (rng.standard_normal((5, 11)) for _ in range(3))
    gamma, beta, vg = (rng.standard_normal(11) for _ in range(3))
    g, b = (gamma, beta) if affine else (None, None)
    _, mean, rstd = R.layer_norm(x, g, b, 1e-3)
    dx, dgamma, dbeta = R.layer_norm_backward(dy, x, g, mean, rstd)
    # central differences of an O(1) function: h^2 truncation plus 1e-16 / h
    assert abs((dx * v).sum() - _difference(lambda z: (R.layer_norm(z, g, b, 1e-3)[0] * dy).sum(), x, v)) < 1e-8
    if affine:
        f = lambda z: (R.layer_norm(x, z, b, 1e-3)[0] * dy).sum()
        assert abs((dgamma * vg).sum() - _difference(f, gamma, vg)) < 1e-8
        f = lambda z: (R.layer_norm(x, g, z, 1e-3)[0] * dy).sum()
        assert abs((dbeta * vg).sum() - _difference(f, beta, vg)) < 1e-8


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("shut", [False, True])
def test_route_gradient_against_differences(renorm, shut):
    rng = np.random.default_rng(4)
    x, v = rng.standard_normal((9, 6)), rng.standard_normal((9, 6))
    valid = np.ones(9, np.uint8)
    if shut:
        x[2, 1:5] = -np.inf
        x[3, :] = -np.inf
        valid[5] = 0
    k, coef = 3, 0.7
    idx, gates, counts, n, mean, loss = R.route(x, k, coef, renorm, valid)
    dgates, dloss = rng.standard_normal((9, k)), 1.3
    dx = R.route_backward(x, idx, counts, n, k, coef, renorm, dgates, dloss, valid)
    f = lambda z: R.route_objective(z, idx, counts, n, k, coef, renorm, dgates, dloss, valid)
    assert abs((dx * np.where(np.isfinite(x), v, 0)).sum() - _difference(f, x, v)) < 1e-8
    if shut:
        assert not dx[3].any() and not dx[5].any() and (idx[3] == -1).all() and (idx[5] == -1).all()
        assert (idx[2] >= 0).sum() == 2 and gates[3].sum() == 0
        assert n == 7 and counts.sum() == (idx >= 0).sum()


def test_balance_loss_is_coef_at_balance():
    x = np.zeros((8, 4))
    x[np.arange(8), np.arange(8) % 4] = 1.0
    loss = R.route(x, 1, 0.3, False)[-1]
    assert abs(loss - 0.3) < 1e-15
