"""Norm and rotation of heads that hold infinities or values whose squares exceed
fp32, in every column and every form of a row's pieces, against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import qk_norm_rope, qk_norm_rope_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, draw, h64

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
