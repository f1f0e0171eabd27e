"""Norm and rotation of heads that hold infinities or values whose squares exceed
fp32, in every column and every form of a row's pieces, against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import qk_norm_rope, qk_norm_rope_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, K, U, draw, h64, half_step, within
from tests.test_heads_gpu import _check_bwd, _check_fwd

pytestmark = pytest.mark.gpu
EPS = 1e-6
INF = float("inf")
# whole pieces, pieces that overlap, angles alone that do not fill theirs, short segments
FORMS = [(64, 64, False), (128, 64, True), (90, 90, False), (90, 90, True), (36, 22, False), (36, 22, True), (80, 40, False),
         (80, 20, True), (127, 0, False), (66, 66, False), (31, 10, False), (20, 4, False), (512, 510, False)]


def _tables(rot, rows):
    cn, sn = R.table(rows, rot)
    c, s = R.token_angles(cn, sn, rot, 1, rows)
    return (None, None, c, s) if rot == 0 else (torch.from_numpy(cn).to(DEV), torch.from_numpy(sn).to(DEV), c, s)


def _same_kind(got, want, what):
    """NaN, infinities with their signs, and finite values at the same places."""
    g = h64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(g), inf) and np.array_equal(g[inf], want[inf]), what


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot,inter", FORMS)
def test_an_infinity_in_every_column(dim, rot, inter, dt):
    """It leaves NaN in its own pair and 0 in the others; in the gradient that comes
    in, infinities in the others."""
    x, dy = (draw((1, dim, 1, dim), i, 1.0, 0.3, DTYPES[dt]).to(DEV) for i in (1, 2))
    g = draw((dim,), 3, 0.2, 1.0).to(DEV)
    cos, sin, c, s = _tables(rot, dim)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    at = torch.arange(dim, device=DEV)
    for v in (INF, -INF):
        bad = x.clone()
        bad[0, at, 0, at] = v
        qk_norm_rope(bad, None, g, None, cos, sin, out, None, interleaved=inter, eps=EPS)
        with np.errstate(invalid="ignore"):
            want = R.qk_norm_rope(h64(bad), h64(g), c, s, rot, inter, EPS)
        _same_kind(out, want, f"{v} in q")
        assert not out[~torch.isnan(out)].any()
        bad = dy.clone()
        bad[0, at, 0, at] = v
        qk_norm_rope_backward(bad, None, x, None, g, None, cos, sin, dx, None, interleaved=inter, eps=EPS)
        with np.errstate(invalid="ignore"):
            want, _ = R.qk_norm_rope_backward(h64(bad), h64(x), h64(g), c, s, rot, inter, EPS)
        _same_kind(dx, want, f"{v} in dq_out")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot,inter", FORMS)
def test_squares_beyond_fp32(dim, rot, inter, dt):
    """Heads of any finite values: from where the sum of their squares exceeds fp32 up
    to the type's highest value, and single such values among ordinary ones."""
    rows = 12
    highest = float(torch.finfo(DTYPES[dt]).max)
    x, dy = (draw((1, rows, 2, dim), i, 1.0, 0.0).to(DEV) for i in (1, 2))
    for i, v in enumerate((1e18, 1e19, 2e19, 1e20, 1e25, 1e31, 1e37)):
        x[0, i] *= v
    x[0, 7], x[0, 8, :, dim // 2] = highest, highest
    x[0, 9, :, dim - 1], x[0, 10, :, 0] = -1e21, -highest
    x, dy = x.to(DTYPES[dt]), dy.to(DTYPES[dt])
    g = draw((dim,), 3, 0.2, 1.0).to(DEV)
    cos, sin, c, s = _tables(rot, rows)
    kw = dict(interleaved=inter, eps=EPS)
    out, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(g)
    qk_norm_rope(x, None, g, None, cos, sin, out, None, **kw)
    _check_fwd(out, x, g, c, s, rot, inter, "out")
    qk_norm_rope_backward(dy, None, x, None, g, None, cos, sin, dx, None, dgamma_q=dg, **kw)
    _check_bwd(dx, dg, dy, x, g, c, s, rot, inter, "dx")
    # the gradients of such heads are small: relative to the largest of a head too, K roundings of the
    # five terms that an element is made of (rows of ordinary directions, r above the smallest numbers)
    want, _ = R.qk_norm_rope_backward(h64(dy), h64(x), h64(g), c, s, rot, inter, EPS)
    err = np.abs(h64(dx) - want)[0, :6].max(-1) / np.abs(want)[0, :6].max(-1)
    assert (err <= 1.01 * half_step(dx.dtype) + 5 * K * U).all()
    qk_norm_rope(x, None, g, None, cos, sin, x, None, **kw)
    assert torch.equal(x, out)


def test_squares_beyond_fp32_and_a_large_eps():
    """An eps that counts beside such squares."""
    x, g = draw((1, 4, 3, 64), 5).to(DEV) * 1e19, draw((64,), 6, 0.2, 1.0).to(DEV)
    dy = draw((1, 4, 3, 64), 7).to(DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    c, s = np.ones((1, 4, 1, 0)), np.zeros((1, 4, 1, 0))
    for eps in (1e30, 1e38, 3e38):
        qk_norm_rope(x, None, g, None, None, None, out, None, eps=eps)
        qk_norm_rope_backward(dy, None, x, None, g, None, None, None, dx, None, eps=eps)
        e = float(np.float32(eps))
        want = R.qk_norm_rope(h64(x), h64(g), c, s, 0, False, e)
        within(out, want, 2 * K * U * np.abs(want), "out")
        want, _ = R.qk_norm_rope_backward(h64(dy), h64(x), h64(g), c, s, 0, False, e)
        r = 1 / np.sqrt((h64(x) ** 2).mean(-1, keepdims=True) + e)
        size = r * (np.abs(h64(dy) * h64(g)) + np.abs(h64(x)) * r * np.abs(h64(dy) * h64(g) * h64(x) * r).mean(-1, keepdims=True))
        assert (np.abs(h64(dx) - want) <= 2 * K * U * size).all()
