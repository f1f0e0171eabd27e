"""The fp64 oracle of the operators at the two ends of a training step against
torch's automatic differentiation in fp64 (CPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ends_ref as R


def _leaf(a):
    return torch.tensor(a, dtype=torch.float64, requires_grad=True)


def _turned(y, c, s, rot, inter):
    """Rotation by complex products, apart from the oracle's form."""
    i, j = (torch.as_tensor(v) for v in R.pairs(rot, inter))
    z = torch.complex(y[..., i], y[..., j]) * torch.complex(torch.tensor(c), torch.tensor(s))
    out = y.clone()
    out[..., i], out[..., j] = z.real, z.imag
    return out


@pytest.mark.parametrize("dim,rot,inter", [(8, 8, False), (8, 4, False), (10, 6, True), (7, 0, False), (6, 6, True)])
def test_heads(dim, rot, inter):
    rng = np.random.default_rng(dim + rot)
    x, dy = rng.standard_normal((2, 5, 3, dim)), rng.standard_normal((2, 5, 3, dim))
    gamma = rng.standard_normal(dim)
    cos, sin = R.table(9, rot)
    c, s = R.token_angles(cos, sin, rot, 2, 5, np.array([[3, 4, -1, 5, 9], [0, 1, 2, 3, 1 << 40]]))
    assert np.all(c[0, 2] == 1) and np.all(s[0, 4] == 0) and np.all(c[1, 4] == 1)
    lx, lg = _leaf(x), _leaf(gamma)
    y = _turned(lx / torch.sqrt((lx ** 2).mean(-1, keepdim=True) + 1e-3) * lg, c, s, rot, inter)
    np.testing.assert_allclose(R.qk_norm_rope(x, gamma, c, s, rot, inter, 1e-3), y.detach(), rtol=1e-12, atol=1e-13)
    want = torch.autograd.grad((y * torch.tensor(dy)).sum(), [lx, lg])
    for got, w in zip(R.qk_norm_rope_backward(dy, x, gamma, c, s, rot, inter, 1e-3), want):
        np.testing.assert_allclose(got, w, rtol=1e-11, atol=1e-12)


def test_turning_keeps_lengths_and_counts_distance():
    cos, sin = R.table(50, 8)
    c, s = R.token_angles(cos, sin, 8, 1, 50)
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal(8), rng.standard_normal(8)
    for inter in (False, True):
        a = R.turn(np.broadcast_to(q, (1, 50, 1, 8)), c, s, 8, inter)[0, :, 0]
        b = R.turn(np.broadcast_to(k, (1, 50, 1, 8)), c, s, 8, inter)[0, :, 0]
        np.testing.assert_allclose((a ** 2).sum(1), (q ** 2).sum(), rtol=1e-6)
        dots = a @ b.T  # depends on the difference of positions only (angles in fp32)
        np.testing.assert_allclose(dots[3, 1], dots[43, 41], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_token_logp(scale):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((9, 13)) * 3
    x[4, 3:9] = -np.inf
    x[5, 2] = 60.0
    x[6] = -np.inf
    t = np.array([0, 12, -100, 13, 1, 2, 3, 5, 6])
    logp, lse = R.token_logp(x, t, scale)
    live = [0, 1, 4, 5, 7, 8]
    lx = _leaf(x)
    ls = torch.log_softmax(lx[live] * scale, 1)
    np.testing.assert_allclose(logp[live], ls.detach()[range(6), t[live]], rtol=1e-9, atol=1e-15)
    np.testing.assert_allclose(lse[live], torch.logsumexp(lx[live] * scale, 1).detach(), rtol=1e-13)
    assert logp[2] == logp[3] == logp[6] == lse[2] == lse[3] == 0 and lse[6] == -np.inf
    assert -1e-15 < logp[5] < 0  # far below the last place of 1
    up = rng.standard_normal(9)
    up[7] = 0.0
    want = torch.zeros_like(lx)
    (g,) = torch.autograd.grad((ls[range(6), t[live]] * torch.tensor(up[live])).sum(), [lx])
    want[live] = g[live]
    np.testing.assert_allclose(R.token_logp_backward(x, t, scale, logp, lse, up), torch.nan_to_num(want), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("old,ref,weighted", [(True, True, True), (True, False, False), (False, True, True)])
def test_policy_loss(old, ref, weighted):
    rng = np.random.default_rng(3)
    n = 400
    lp = -np.exp(rng.standard_normal(n))
    ol = lp + rng.standard_normal(n) * 0.3 if old else None
    rf = lp + rng.standard_normal(n) * 0.3 if ref else None
    adv = rng.standard_normal(n)
    adv[:5] = 0
    w = rng.random(n) * (rng.random(n) < 0.8) if weighted else None
    loss, terms, g = R.policy_loss(lp, ol, rf, adv, w, 0.2, 0.3, 0.1, 1.5)
    l = _leaf(lp)
    a = torch.tensor(adv)
    ratio = torch.exp(l - (l.detach() if ol is None else torch.tensor(ol)))
    if ol is None:
        pg = -a * ratio
    else:
        pg = -torch.minimum(ratio * a, ratio.clamp(0.8, 1.3) * a)
    kl = torch.zeros(n, dtype=torch.float64)
    if ref:
        u = torch.tensor(rf) - l
        kl = torch.exp(u) - u - 1
    wt = torch.ones(n, dtype=torch.float64) if w is None else torch.tensor(w)
    f = (wt * (pg + 0.1 * kl)).sum()
    assert abs(loss - float(f)) < 1e-11 and abs(terms[0] + 0.1 * terms[1] - loss) < 1e-12
    (want,) = torch.autograd.grad(1.5 * f, [l])
    np.testing.assert_allclose(g, want, rtol=1e-10, atol=1e-13)
    if old:
        assert 0 < terms[2] < (n if w is None else w.sum())


@pytest.mark.parametrize("average,masked,ref", [(False, False, True), (True, True, True), (True, False, False)])
def test_preference_loss(average, masked, ref):
    rng = np.random.default_rng(4)
    p = 5
    off = np.array([2, 5, 5, 9, 20, 21, 30, 31, 31, 44, 50])
    n = 53
    lp, rf = -np.exp(rng.standard_normal(n)), -np.exp(rng.standard_normal(n)) if ref else None
    v = (rng.random(n) < 0.7) if masked else None
    w = rng.random(p)
    w[2] = 0
    before = np.full(n, 9.0)
    loss, rewards, g = R.preference_loss(lp, rf, v, off, w, 0.3, 0.2, 0.1, average, 0.7, before)
    l = _leaf(lp)
    d = l if rf is None else l - torch.tensor(rf)
    if masked:
        d = torch.where(torch.tensor(v), d, torch.zeros(()).double())
    sums = []
    for s in range(2 * p):
        run = d[off[s]:off[s + 1]]
        cnt = run.numel() if not masked else int(v[off[s]:off[s + 1]].sum())
        sums.append(0.3 * run.sum() / (max(cnt, 1) if average else 1))
    m = torch.stack(sums[:p]) - torch.stack(sums[p:]) - 0.2
    f = (torch.tensor(w) * -(0.9 * torch.nn.functional.logsigmoid(m) + 0.1 * torch.nn.functional.logsigmoid(-m))).sum()
    assert abs(loss - float(f)) < 1e-12
    np.testing.assert_allclose(rewards, [float(x) for x in sums], rtol=1e-11, atol=1e-14)
    (want,) = torch.autograd.grad(0.7 * f, [l])
    np.testing.assert_allclose(g[2:50], want[2:50], rtol=1e-10, atol=1e-14)
    assert np.all(g[:2] == 9) and np.all(g[50:] == 9)
