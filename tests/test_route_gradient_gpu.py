"""GPU router gradient where its terms are far smaller than what they are the
difference of, or where what reaches it is not finite."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import route, route_backward
from oracle import ops_ref as R
from tests.ops_helpers import DEV, DTYPES, K, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu


def _forward(x, k, renorm, valid=None):
    rows, experts = x.shape
    idx, gates = torch.empty(rows, k, dtype=torch.int32, device=DEV), torch.empty(rows, k, device=DEV)
    counts, n = torch.empty(experts, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    route(x, idx, gates, counts, n, torch.empty(1, device=DEV), coef=0.1, renorm=renorm, valid=valid)
    return idx, counts, n


def _gradient(x, idx, dgates, counts, n, coef, renorm):
    """(dlogits, bound) in fp64 from differences to the token's most probable
    expert, whose p is 1 less the others': dlogit = p (dp - sum p dp) with
    dp - dp_top in the place of dp, and likewise for renormalised gates.  The
    bound counts roundings of what those differences are taken of; the
    exponential's argument has one of the size of the distance."""
    rows, e = x.shape
    r, k = np.arange(rows), idx.shape[1]
    top = x.argmax(1)
    z = np.exp(x - x[r, top][:, None])
    p = z / z.sum(1, keepdims=True)
    rel = 2 * (K + np.ptp(x, axis=1)[:, None]) * U
    dg, at = np.asarray(dgates, float), np.asarray(idx)
    mag = np.abs(dg)
    if renorm:
        q = np.take_along_axis(p, at, 1)
        s = q.sum(1, keepdims=True)
        best = q.argmax(1)
        dg = dg - dg[r, best][:, None]
        mag = np.abs(dg)
        mid, mmid = ((v * q / s).sum(1, keepdims=True) for v in (dg, mag))
        dg, mag = (dg - mid) / s, (mag + mmid) / s
    c = np.asarray(counts, float)
    bal = coef * (e * c - c.sum()) / (k * n ** 2)  # less a constant, which sum p = 1 takes out
    dp, m = np.tile(bal, (rows, 1)), np.tile(np.abs(bal), (rows, 1))
    for j in range(k):
        dp[r, at[:, j]] += dg[:, j]
        m[r, at[:, j]] += mag[:, j]
    dp, m = dp - dp[r, top][:, None], m + m[r, top][:, None]
    m[r, top] = 0
    want = p * (dp - (p * dp).sum(1, keepdims=True))
    return want, rel * p * (m + (p * m).sum(1, keepdims=True))


@pytest.mark.parametrize("experts,k", [(8, 4), (24, 4), (64, 4), (512, 4), (1000, 16)])
def test_counts_of_many_ranks(experts, k):
    """Counts summed over ranks: each fits its type, their sum k n need not.
    Near balance their differences are what matters."""
    n = (1 << 31) - 5
    counts = k * n // experts + np.random.default_rng(experts).integers(-1000, 1000, experts)
    assert counts.max() < 1 << 31 < counts.sum()
    x = draw((50, experts), 9).to(DEV)
    idx, _, _ = _forward(x, k, False)
    dx = torch.empty_like(x)
    route_backward(x, idx, torch.tensor(counts, dtype=torch.int32, device=DEV),
                   torch.tensor([n], dtype=torch.int32, device=DEV), dx, coef=float(n), renorm=False)
    want, bound = _gradient(h64(x), idx.cpu().numpy(), np.zeros((50, k)), counts, n, float(np.float32(n)), False)
    within(dx, want, bound + U * (np.abs(want) + bound), "dlogits")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("experts,k", [(8, 2), (24, 2), (64, 4), (300, 8)])
@pytest.mark.parametrize("dloss", [float("inf"), float("-inf"), float("nan")])
def test_overflowed_loss_scale_leaves_padding_at_zero(experts, k, dt, dloss):
    """A gradient of the loss that is not finite reaches the tokens with a
    choice only."""
    rows = 150
    x = draw((rows, experts), 3, 1.0, 0.0, DTYPES[dt]).to(DEV)
    x[20:30] = float("-inf")                     # every expert shut off
    valid = torch.ones(rows, dtype=torch.uint8, device=DEV)
    valid[40:55] = 0
    valid[149] = 0
    idx, counts, n = _forward(x, k, True, valid)
    x[40:55] = float("nan")
    dgates = draw((rows, k), 7).to(DEV)
    for dg in (dgates, None):
        dx = torch.full_like(x, 5.0)
        route_backward(x, idx, counts, n, dx, dgates=dg, dloss=torch.tensor([dloss], device=DEV), coef=0.1, valid=valid)
        none = torch.zeros(rows, dtype=torch.bool, device=DEV)
        none[20:30] = none[40:55] = none[149] = True
        assert (dx[none] == 0).all()
        assert not torch.isfinite(dx[~none]).any()




@pytest.mark.parametrize("coef", [0.0, 0.3])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("experts,k", [(2, 1), (2, 2), (8, 1), (8, 2), (16, 2), (24, 3), (64, 6), (100, 1), (128, 8),
                                       (256, 8), (512, 4), (1000, 2)])
def test_confident_tokens(experts, k, dt, renorm, coef):
    """One expert far above the rest: the gradients are those of the rest's
    small probabilities, to a relative error."""
    gaps = np.array([8.0, 12.0, 13.0, 14.0, 15.0, 16.0, 17.0, 18.0, 20.0, 24.0, 40.0, 60.0])
    rows = len(gaps)
    x = draw((rows, experts), experts + k, 0.3)
    top = torch.from_numpy(np.random.default_rng(k).integers(0, experts, rows))
    x[torch.arange(rows), top] = torch.from_numpy(gaps).float() + experts ** 0.1
    x = x.to(DTYPES[dt]).to(DEV)
    idx, counts, n = _forward(x, k, renorm)
    dgates = draw((rows, k), 7).to(DEV)
    dx = torch.full_like(x, 5.0)
    route_backward(x, idx, counts, n, dx, dgates=dgates, coef=coef, renorm=renorm)
    want, bound = _gradient(h64(x), idx.cpu().numpy(), h64(dgates), counts.cpu().numpy(), rows, coef, renorm)
    within(dx, want, bound + half_step(x.dtype) * (np.abs(want) * (1 + 1e-6) + bound), "dlogits")
    # the oracle's plain formula in fp64 agrees as far as its own cancellation allows
    plain = R.route_backward(h64(x), idx.cpu().numpy(), counts.cpu().numpy(), rows, k, coef, renorm, h64(dgates), 1.0)
    assert (np.abs(plain - want) <= 1e-12 * (np.abs(h64(dgates)).max() + coef * experts) * 4 * experts).all()
