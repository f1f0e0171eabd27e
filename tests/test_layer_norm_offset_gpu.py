"""GPU layer norm of rows whose common offset is large against their spread:
the statistics have to be those of the row, not of the rounding of its mean."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import (dropout_add_layer_norm, dropout_add_layer_norm_backward, layer_norm,
                                  layer_norm_backward)
from oracle import ops_ref as R
from tests.ops_helpers import DEV, DTYPES, K, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu
EPS = 1e-5
# around the changes of the threads and vectors a row takes, whole and ragged
WIDTHS = [5, 37, 120, 300, 777, 1000, 1536, 1537, 4096, 6001, 8192, 12296, 20000, 20003, 32768]


def _rows(cols, dt):
    """Constants whose sums round, a spread far below the offset, one element
    off, one far larger than the rest, and ordinary rows."""
    x = draw((10, cols), cols)
    x[0], x[1], x[2], x[3] = 1000.1, 10000.1, 12345.67, -0.3
    x[4] = x[4] * 1e-3 + 1000.1
    x[5] = x[5] * 1e-2 - 12345.67
    x[6] = 1000.0
    x[6, cols // 2] = 1004.0
    x[7, 0] = 1e4
    x[8] = x[8] + 100
    return x.to(DTYPES[dt]).to(DEV)


def _bounds(x, gamma, beta, y, mean, rstd, dtype):
    """(y, mean, rstd).  A sum over a row has at most K roundings in a chain (40
    additions in a thread, 6 across a wave, 15 across the waves, a division).
    The first mean is off by `first`; the deviations from it are rounded once,
    their mean (K roundings of numbers the size of the deviations) and its
    subtraction once more.  So no rounding is of the size of the offset but
    that of the stored mean, and the second-order ones of `first`.  A row whose
    mean is within two deviations has the first mean alone."""
    d, first = np.abs(x - mean[:, None]), K * U * np.abs(x).mean(1)[:, None]
    shift = K * U * (d.mean(1)[:, None] + first)
    shift = shift + np.where(np.abs(mean[:, None]) <= 2.01 * np.sqrt((d ** 2).mean(1))[:, None], first, 0)
    dev = 1.01 * (U * (2 * d + first) + shift)
    rel = K * U + (2 * d * dev + dev ** 2).mean(1) * rstd ** 2
    g = 1.0 if gamma is None else np.abs(gamma)
    b = 0.0 if beta is None else np.abs(beta)
    by = half_step(dtype) * np.abs(y) * (1 + 1e-6) + 1.01 * (dev + d * (rel[:, None] + 4 * U)) * rstd[:, None] * g \
        + 2 * U * (np.abs(y) + b)
    # a constant row's y is a rounding error, stored with one of its own
    by = by + half_step(dtype) * by
    return by, U * np.abs(mean) * (1 + 1e-6) + shift[:, 0], (rel + 4 * U) * rstd


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_offsets(cols, dt, affine):
    x = _rows(cols, dt)
    gamma = draw((cols,), 1, 0.2, 1.0).to(DEV) if affine else None
    beta = draw((cols,), 2, 0.2).to(DEV) if affine else None
    y, mean, rstd = torch.empty_like(x), torch.empty(10, device=DEV), torch.empty(10, device=DEV)
    layer_norm(x, gamma, beta, y, mean=mean, rstd=rstd, eps=EPS)
    xs = h64(x)
    g, b = (None if t is None else h64(t) for t in (gamma, beta))
    # the fp64 mean of a constant is off by its own roundings, far below the bounds
    wy, wm, wr = R.layer_norm(xs, g, b, EPS)
    by, bm, br = _bounds(xs, g, b, wy, wm, wr, x.dtype)
    within(mean, wm, bm, "mean")
    within(rstd, wr, br, "rstd")
    within(y, wy, by, "y")
    # the fused pass on the same rows (everything dropped: h is the residual)
    h, y2, m2, r2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(mean), torch.empty_like(rstd)
    dropout_add_layer_norm(torch.zeros_like(x), x, gamma, beta, h, y2, mean=m2, rstd=r2, eps=EPS, p=1.0, seed=3)
    for got, want in ((h, x), (y2, y), (m2, mean), (r2, rstd)):
        assert torch.equal(got, want)


def test_tiny_eps():
    """With eps far below the spread of an offset row the variance is that of
    the spread: a few elements of many that differ by one step of the type."""
    cols, eps = 8192, 1e-14
    x = torch.full((3, cols), 1000.1, device=DEV)
    x[0, ::64] = torch.nextafter(x[0, 0], torch.tensor(2e3, device=DEV))
    x[1, 5::1024] = 1000.2
    x[2, ::2] = torch.nextafter(x[2, 0], torch.tensor(0.0, device=DEV))
    y, mean, rstd = torch.empty_like(x), torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    layer_norm(x, None, None, y, mean=mean, rstd=rstd, eps=eps)
    xs = h64(x)
    wy, wm, wr = R.layer_norm(xs, None, None, eps)
    by, bm, br = _bounds(xs, None, None, wy, wm, wr, x.dtype)
    within(mean, wm, bm, "mean")
    within(rstd, wr, br, "rstd")
    within(y, wy, by, "y")


@pytest.mark.parametrize("rows", [3, 600])
@pytest.mark.parametrize("cols", [3, 8, 13, 40, 100])
def test_gradient_of_huge_constant_rows(cols, rows):
    """Constant rows so large that mean * rstd overflows: their xh is 0, so
    dx = rstd (g - mean(g)), whatever threads hold no element of the row."""
    x = torch.full((rows, cols), 2.0 ** 121, device=DEV)
    x[1] = -(2.0 ** 121)
    dy = draw((rows, cols), 5).to(DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    layer_norm(x, None, None, y, mean=mean, rstd=rstd, eps=EPS)
    assert torch.equal(mean, x[:, 0].contiguous()) and not y.any()
    assert torch.isinf(mean * rstd).all()
    dx, dg, db = torch.empty_like(x), torch.full((cols,), 5.0, device=DEV), torch.empty(cols, device=DEV)
    layer_norm_backward(dy, x, None, mean, rstd, dx, dgamma=dg, dbeta=db)
    g, r = h64(dy), h64(rstd)[:, None]
    want = r * (g - g.mean(1, keepdims=True))
    within(dx, want, U * np.abs(want) * (1 + 1e-6) + K * U * r * (np.abs(g) + np.abs(g).mean(1, keepdims=True)), "dx")
    assert not dg.any()
    dx2, dres = torch.empty_like(x), torch.empty_like(x)
    dropout_add_layer_norm_backward(dy, x, None, mean, rstd, dx2, dres, p=0.0, seed=1)
    assert torch.equal(dres, dx) and torch.equal(dx2, dx)
