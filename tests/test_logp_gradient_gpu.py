"""The gradient of the log-probabilities against that of the logits themselves in
fp64 (not of the lse that the forward pass rounded): rows far from 0, at the
type's lowest value, beyond fp32 when scaled, and with unlikely targets."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import token_logp, token_logp_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu
INF = float("inf")
NEAR = 64.0  # a statistic of at most this size is used as it was rounded


def _bounds(x, t, scale, dlogp, want, dtype):
    """Elementwise bounds.  A probability comes from a statistic (lse where it is at
    most 64, else logp where it is, else the logarithm of the row's sum formed
    again) and the difference to it.  The statistic has its own rounding, and the
    error of the sum: its logarithm's two steps, the terms' (three roundings of their distance to the maximum, on
    average over the terms) and its additions', at most vocab / 64 in a thread, each
    with a rescaling, and 20 joins.  logp also has the three roundings of the
    target's distance to the maximum, and the difference to the target's logit
    one of its own.  The distance of a word to lse is rounded four times before
    the exponential, which adds two; a few products follow.  The target's own
    gradient is off by that of logp, relative to it where it is next to 0."""
    b = np.zeros_like(x)
    chain = 1.25 * x.shape[1] / (64 if x.shape[1] <= 2048 else 256) + 40
    g = np.abs(scale * dlogp)
    for i, at in enumerate(t):
        if not 0 <= at < x.shape[1] or dlogp[i] == 0 or np.all(x[i] == -INF):
            continue
        z = x[i] * scale
        d = z.max() - z
        e = np.exp(-d)
        total, rest = e.sum(), np.delete(e, at).sum()
        far = np.where(e > 0, d, 0.0)
        mean = (e * far).sum() / total
        mean_rest = np.delete(e * far, at).sum() / max(rest, 1e-300)
        lse, logp = z.max() + np.log(total), -d[at] - np.log(total)
        stat = abs(lse) if abs(lse) <= NEAR else 5 * abs(logp) + 6 if abs(logp) <= NEAR else np.log(total)
        away = np.where(e > 0, d + np.log(total), 0.0)
        b[i] = (4 * away + 3 * mean + chain + stat + 4 * np.log(total) + 16) * U * np.abs(want[i])
        b[i] += half_step(dtype) * np.abs(want[i]) * (1 + 1e-6) + g[i] * 2.0 ** -126 * 1.01
        dl = 3 * mean_rest + chain + 4 * np.log(total) + 12 + (3 * d[at] + abs(logp) if abs(logp) < 200 else 0)
        if rest < e[at]:
            own = dl * np.abs(want[i, at])
        else:
            own = dl * g[i] * np.exp(logp) + 3 * np.abs(want[i, at])
        b[i, at] = half_step(dtype) * np.abs(want[i, at]) * (1 + 1e-6) + (own + 6 * np.abs(want[i, at])) * U \
            + g[i] * 2.0 ** -126
    return b


def _check(x, t, scale, d, rows=None, what=""):
    """Forward, gradient into another tensor and in place, both against the oracle."""
    logp, lse = torch.empty(x.shape[0], device=DEV), torch.empty(x.shape[0], device=DEV)
    token_logp(x, t, logp, lse, scale=scale)
    dx = torch.full_like(x, 5.0)
    token_logp_backward(x, t, logp, lse, d, dx, scale=scale)
    part = slice(None) if rows is None else rows
    xs, ts, sc, ds = h64(x[part]), t[part].cpu().numpy(), float(np.float32(scale)), h64(d[part])
    want = R.token_logp_gradient(xs, ts, sc, ds)
    within(dx[part], want, _bounds(xs, ts, sc, ds, want, x.dtype), f"dlogits {what}")
    y = x.clone()
    token_logp_backward(y, t, logp, lse, d, y, scale=scale)
    assert torch.equal(y, dx), f"in place {what}"
    return logp, lse, dx


def _case(rows, vocab, dt, seed, offset=0.0):
    """Logits around an offset, a fifth of the targets likely ones, one in ten none."""
    x = draw((rows, vocab), seed, 3.0, offset, DTYPES[dt]).to(DEV)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    t = torch.from_numpy(rng.integers(0, vocab, rows))
    for i in range(0, rows, 5):
        x[i, t[i]] = offset + 25.0
    t[3::10] = -100
    return x, t.to(DEV), draw((rows,), seed + 2).to(DEV)


VOCABS = [1, 5, 60, 100, 200, 256, 500, 1000, 2048, 2500, 8200, 50021]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_offsets(vocab, dt):
    for offset in (0.0, 70.0, -70.0, 1e3, -1e3, 1e5, -1e6):
        x, t, d = _case(21, vocab, dt, vocab, offset)
        _check(x, t, 1.0, d, what=f"offset {offset}")
        _check(x, t, 1.25, d, what=f"offset {offset}, scaled")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", VOCABS[1:])
def test_masked_rows(vocab, dt):
    """Rows at a mask's finite floor or at the type's lowest value, whose scaled
    logits exceed fp32 too; rows of -inf; targets that cannot be, far from 0 or not."""
    lowest = torch.finfo(DTYPES[dt]).min
    x, t, d = _case(24, vocab, dt, 3 + vocab)
    x[1], t[1] = lowest, 2
    x[2], t[2] = -1e9, 0
    x[4], t[4] = -INF, 1
    x[5], t[5] = -INF, vocab - 1
    x[5, vocab - 1] = lowest            # the target alone is left
    x[6, ::2], t[6] = lowest, 3
    x[7] += 1e4
    t[7] = 2
    x[7, 2] = -INF                      # it cannot be, and lse is large
    x[8], t[8] = -INF, 1
    x[8, 3] = 1.0                       # another word alone is left
    x[9], t[9] = lowest, 4
    x[9, 4] = -INF                      # nor where lse is beyond fp32
    x[10], t[10] = -lowest, 2           # at the highest value
    x[11], t[11] = -lowest, 1
    x[11, 1] = -INF
    x[12, 2:], t[12] = lowest, 4        # a masked target among two words
    x[14], d[14] = float("nan"), 0.0    # not read
    for scale in (1.0, 1.25, 0.5):
        logp, lse, dx = _check(x, t, scale, d, rows=[i for i in range(24) if i != 14], what=f"scale {scale}")
        assert not dx[4].any() and not dx[14].any()
        if dt == "f32":                 # every word of a row of equal ones has the same part
            sc = float(np.float32(scale))
            for i in (1, 2, 10):
                own = -float(d[i]) * sc / vocab
                others = torch.cat([dx[i, : int(t[i])], dx[i, int(t[i]) + 1 :]])
                assert ((others - own).abs() <= 1e-4 * abs(own)).all(), (i, scale)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [7, 100, 250, 1000, 3001, 40000])
def test_large_scales_and_unlikely_targets(vocab, dt):
    """Both lse and logp are large."""
    for scale in (1e4, 1e8, 1e30):
        x, t, d = _case(21, vocab, dt, 5 + vocab)
        _check(x, t, scale, d / np.float32(scale), what=f"scale {scale}")
    x, t, d = _case(21, vocab, dt, 6 + vocab, 1e3)
    for i in range(21):
        if t[i] >= 0:
            x[i, t[i]] = 1e3 - 10.0 ** (i / 6)
    _check(x, t, 1.0, d, what="unlikely")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_values(dt):
    """Rows with NaN or +inf, whole ones too, have NaN, others are as they were."""
    for vocab in (90, 200, 1000, 30000):
        x, t, d = _case(12, vocab, dt, 7, 1e3)
        t[3] = 0
        _, _, want = _check(x, t, 1.0, d)
        y = x.clone()
        y[2], y[5, 4], y[7, 1], y[8, t[8]], y[9, t[9]] = float("nan"), float("nan"), INF, float("nan"), INF
        logp, lse = torch.empty(12, device=DEV), torch.empty(12, device=DEV)
        token_logp(y, t, logp, lse)
        for out in (torch.empty_like(x), y):
            token_logp_backward(y, t, logp, lse, d, out)
            bad = torch.zeros(12, dtype=torch.bool, device=DEV)
            bad[[2, 5, 7, 8, 9]] = True
            assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_rows_far_from_zero(dt):
    """Rows of each kind among many, strided and in place, and logits beyond the caches."""
    for rows, vocab in ((5000, 100), (5000, 130), (700, 3001), (260, 20000)):
        x, t, d = _case(rows, vocab, dt, 9)
        x[::3] += 300.0
        for i in range(0, rows, 11):
            if t[i] >= 0:
                x[i, t[i]] -= 200.0
        part = list(range(0, rows, max(rows // 60, 1))) + [rows - 1]
        _, _, dx = _check(x, t, 0.9, d, rows=part)
        buf = torch.full((rows * (vocab + 3) + 1,), 3.0, dtype=x.dtype, device=DEV)
        v = buf[1:].view(rows, vocab + 3)[:, :vocab]
        v.copy_(x)
        logp, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        token_logp(v, t, logp, lse, scale=0.9)
        token_logp_backward(v, t, logp, lse, d, v, scale=0.9)
        assert torch.equal(v, dx)
        v.fill_(3.0)
        assert (buf == 3.0).all()
    vocab = 30011
    rows = (260 << 20) // (vocab * x.element_size())
    few, t, d = _case(64, vocab, dt, 10, 500.0)
    x = few.repeat(rows // 64 + 1, 1)[:rows].contiguous()
    t, d = t.repeat(rows // 64 + 1)[:rows].contiguous(), d.repeat(rows // 64 + 1)[:rows].contiguous()
    _check(x, t, 1.0, d, rows=list(range(20)) + [rows - 1])


def test_gradient_against_differences():
    rows, vocab, scale = 9, 31, 1.5
    x, t, d = _case(rows, vocab, "f32", 21, 1e3)
    _, _, dx = _check(x, t, scale, d)
    v = h64(draw((rows, vocab), 24))
    f = lambda z: (R.token_logp(z, t.cpu().numpy(), scale)[0] * h64(d)).sum()
    num = (f(h64(x) + 1e-4 * v) - f(h64(x) - 1e-4 * v)) / 2e-4
    assert abs((h64(dx) * v).sum() - num) <= 1e-6 + 400 * U * np.abs(v).sum() * np.abs(h64(d)).max() * scale
