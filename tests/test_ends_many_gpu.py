"""More rows than one launch has workgroups for, so that the kernels' loops over
what is left take a second round, and many pairs of answers."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import qk_norm_rope, token_logp, token_logp_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, draw, h64, within
from tests.test_logp_gpu import _check
from tests.test_logp_gradient_gpu import _bounds
from tests.test_losses_gpu import _check_pref, _pref

pytestmark = pytest.mark.gpu


def _rows(rows, vocab, dt, seed):
    """Random rows repeated (a fifth without a target, some far from 0)."""
    few = 4099
    x = draw((few, vocab), seed, 3.0, 0.0, DTYPES[dt]).to(DEV)
    x[5::7] += 500.0
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    t = torch.from_numpy(rng.integers(0, vocab, few))
    t[rng.random(few) < 0.2] = -100
    d = draw((few,), seed + 2).to(DEV)
    n = rows // few + 1
    return x.repeat(n, 1)[:rows].contiguous(), t.to(DEV).repeat(n)[:rows].contiguous(), d.repeat(n)[:rows].contiguous(), few


@pytest.mark.parametrize("vocab,dt,border", [(9, "bf16", 65535 * 16), (130, "bf16", 65535 * 8), (300, "bf16", 65535 * 4),
                                             (20, "f32", 65535 * 16), (100, "f32", 65535 * 8), (257, "f32", 65535 * 4),
                                             (2049, "bf16", 65535), (1025, "f32", 65535)])
def test_gradient_rows_beyond_one_launch(vocab, dt, border):
    """The rows' dimension of the grid ends at 65535 workgroups of 16, 8, 4 rows or one."""
    rows = border + 1013
    x, t, d, few = _rows(rows, vocab, dt, vocab)
    logp, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    token_logp(x, t, logp, lse)
    dx = torch.full_like(x, 5.0)
    token_logp_backward(x, t, logp, lse, d, dx)
    # a row has the same bits wherever it stands
    for out in (dx, logp, lse):
        for at in range(few, rows, 64 * few):
            n = min(few, rows - at)
            assert torch.equal(out[at:at + n], out[:n])
        last = rows // few * few
        assert torch.equal(out[last:], out[: rows - last])
    part = torch.cat([torch.arange(0, few, 131, device=DEV), torch.tensor([border - 1, border, border + 1, rows - 1], device=DEV)])
    xs, ts, ds = h64(x[part]), t[part].cpu().numpy(), h64(d[part])
    want = R.token_logp_gradient(xs, ts, 1.0, ds)
    within(dx[part], want, _bounds(xs, ts, 1.0, ds, want, x.dtype), "dlogits")
    token_logp_backward(x, t, logp, lse, d, x)
    assert torch.equal(x, dx)


def test_forward_rows_beyond_one_launch():
    """2^20 workgroups of 64 rows."""
    rows, vocab = (1 << 26) + 70001, 2
    x, t, _, few = _rows(rows, vocab, "bf16", 3)
    logp, lse = torch.full((rows,), 7.0, device=DEV), torch.full((rows,), 7.0, device=DEV)
    token_logp(x, t, logp, lse)
    _check(x[:few], t[:few], 1.0, logp[:few], lse[:few])
    last = rows // few * few
    for out in (logp, lse):
        assert torch.equal(out[:last].view(-1, few), out[:few].expand(last // few, few))
        assert torch.equal(out[last:], out[: rows - last])


def test_heads_beyond_one_launch():
    """2^20 workgroups of 64 heads of 16."""
    tokens, heads = (1 << 21) + 3001, 32
    q = draw((1, 997, heads, 16), 1, 1.3, 0.2, torch.bfloat16).to(DEV)
    n = tokens // 997 + 1
    cn, sn = R.table(97, 16)
    cos, sin = torch.from_numpy(cn).to(DEV), torch.from_numpy(sn).to(DEV)
    pos = (torch.arange(997, device=DEV) % 97).repeat(n)[:tokens].contiguous()
    many = q.repeat(1, n, 1, 1)[:, :tokens].contiguous()
    few, out = torch.empty_like(q), torch.full_like(many, 3.0)
    qk_norm_rope(q, None, None, None, cos, sin, few, None, positions=pos[:997])
    qk_norm_rope(many, None, None, None, cos, sin, out, None, positions=pos)
    last = tokens // 997 * 997
    assert torch.equal(out[:, :last].view(-1, 997, heads, 16), few.expand(last // 997, 997, heads, 16))
    assert torch.equal(out[:, last:], few[:, : tokens - last])


@pytest.mark.parametrize("pairs,mean", [(100003, 2), (3001, 700)])
def test_many_pairs(pairs, mean):
    rng = np.random.Generator(np.random.PCG64(pairs))
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(rng.integers(0, 2 * mean + 1, 2 * pairs))])).to(DEV)
    n = int(off[-1])
    lp = -torch.exp(draw((n,), 1, 1.5, -1.5)).to(DEV)
    rf = (lp + draw((n,), 2, 0.1).to(DEV)).clamp(max=0)
    v = draw((n,), 3).to(DEV) > -0.5
    w = torch.from_numpy(rng.random(pairs, dtype=np.float32) / pairs).to(DEV)
    kw = dict(beta=0.1, margin=0.2, smoothing=0.1)
    out = _pref(lp, off, rf, v, w, **kw)
    _check_pref(lp, off, rf, v, w, out, **kw)
