"""Plain fp64 CPU oracle for the operators at the two ends of a training step:
the norm and rotation of query and key heads, token log-probabilities, the
clipped policy loss and the preference loss.

TEST INFRASTRUCTURE ONLY, like muon_ref: only the test suite may import it,
and it imports nothing from the product path.  The formulas are those that
include/muon.h states; every operation is a fp64 NumPy expression.
"""
from __future__ import annotations

import numpy as np


# ---- norm and rotation of heads ------------------------------------------------

def table(rows, rot, base=10000.0):
    """(cos, sin), [rows, rot / 2], in fp32 as a caller keeps them."""
    f = base ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(rows)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def token_angles(cos, sin, rot, batch, tokens, positions=None):
    """Angles of every token, [batch, tokens, 1, rot / 2]; (1, 0) for a token
    whose row does not exist."""
    n = cos.shape[0] if rot else 0
    pos = np.broadcast_to(np.arange(tokens) if positions is None else positions, (batch, tokens))
    ok = (pos >= 0) & (pos < n)
    c, s = np.ones((batch, tokens, rot // 2)), np.zeros((batch, tokens, rot // 2))
    if rot:
        c[ok], s[ok] = cos[pos[ok]], sin[pos[ok]]
    return c[:, :, None], s[:, :, None]


def pairs(rot, interleaved):
    """Columns of the pairs' first and second elements."""
    if interleaved:
        return np.arange(0, rot, 2), np.arange(1, rot, 2)
    return np.arange(rot // 2), np.arange(rot // 2, rot)


def turn(y, c, s, rot, interleaved):
    i, j = pairs(rot, interleaved)
    out = y.copy()
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def qk_norm_rope(x, gamma, c, s, rot, interleaved, eps):
    """x [batch, tokens, heads, dim]; c, s as token_angles gives them."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r
    if gamma is not None:
        y = y * gamma
    return turn(y, c, s, rot, interleaved)


def qk_norm_rope_backward(dy, x, gamma, c, s, rot, interleaved, eps):
    """(dx, dgamma)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    g = turn(dy, c, -s, rot, interleaved)
    dgamma = (g * xh).reshape(-1, x.shape[-1]).sum(0)
    if gamma is not None:
        g = g * gamma
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), dgamma


# ---- token log-probabilities -----------------------------------------------------

def token_logp(x, targets, scale):
    """(logp, lse) of logits x [tokens, vocab]."""
    rows, vocab = x.shape
    logp, lse = np.zeros(rows), np.zeros(rows)
    for i in range(rows):
        t = int(targets[i])
        if not 0 <= t < vocab:
            continue
        z = x[i] * scale
        m = z.max()
        if m == -np.inf:
            lse[i] = -np.inf
            continue
        with np.errstate(invalid="ignore"):
            e = np.exp(z - m)
        rest = np.delete(e, t).sum()
        lse[i] = m + np.log(e[t] + rest)
        with np.errstate(divide="ignore"):
            logp[i] = -np.log1p(rest / e[t]) if e[t] > rest else (z[t] - m) - np.log(e[t] + rest)
    return logp, lse


def token_logp_gradient(x, targets, scale, dlogp):
    """The gradient of sum(dlogp * logp) by the logits, from the logits alone."""
    out = np.zeros_like(x)
    for i in range(x.shape[0]):
        t = int(targets[i])
        if not 0 <= t < x.shape[1] or dlogp[i] == 0 or np.all(x[i] == -np.inf):
            continue
        z = x[i] * scale
        e = np.exp(z - z.max())
        out[i] = -scale * dlogp[i] * e / e.sum()
        out[i, t] = scale * dlogp[i] * np.delete(e, t).sum() / e.sum()
    return out


def token_logp_backward(x, targets, scale, logp, lse, dlogp):
    """The same from given logp and lse: they are taken as exact."""
    out = np.zeros_like(x)
    for i in range(x.shape[0]):
        t = int(targets[i])
        if not 0 <= t < x.shape[1] or dlogp[i] == 0 or lse[i] == -np.inf:
            continue
        p = np.exp(x[i] * scale - lse[i])
        out[i] = -scale * dlogp[i] * p
        out[i, t] = -scale * dlogp[i] * np.expm1(logp[i])
    return out


# ---- losses ------------------------------------------------------------------------

def policy_loss(logp, old, ref, adv, weight, low, high, beta, dloss=1.0):
    """(loss, (policy, KL, clipped), dlogp); old, ref, weight may be None."""
    n = logp.shape[0]
    w = np.ones(n) if weight is None else weight
    dlogp, pg_sum, kl_sum, cut_sum = np.zeros(n), 0.0, 0.0, 0.0
    for i in np.nonzero(w != 0)[0]:
        d = 0.0 if old is None else logp[i] - old[i]
        a = adv[i]
        with np.errstate(over="ignore"):
            ratio = np.exp(d)
        lo, hi = 1.0 - low, 1.0 + high
        with np.errstate(divide="ignore"):
            cut = (a > 0 and d > np.log(hi)) or (a < 0 and d < np.log(lo))
        gain = 0.0 if a == 0 else a * ratio
        pg = -a * (hi if a > 0 else lo) if cut else -gain
        kl, dkl = 0.0, 0.0
        if ref is not None:
            u = ref[i] - logp[i]
            with np.errstate(over="ignore"):
                kl, dkl = np.expm1(u) - u, -np.expm1(u)
        pg_sum += w[i] * pg
        kl_sum += w[i] * kl
        cut_sum += w[i] * cut
        dlogp[i] = dloss * w[i] * ((0.0 if cut else -gain) + (beta * dkl if beta else 0.0))
    return pg_sum + (beta * kl_sum if beta else 0.0), (pg_sum, kl_sum, cut_sum), dlogp


def _softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def preference_loss(logp, ref, valid, offsets, weight, beta, margin, smoothing, average, dloss=1.0, dlogp=None):
    """(loss, rewards, dlogp); dlogp given: what it held before."""
    n, p = logp.shape[0], (len(offsets) - 1) // 2
    v = np.ones(n, bool) if valid is None else np.asarray(valid) != 0
    d = np.where(v, logp, 0.0) - (0.0 if ref is None else np.where(v, ref, 0.0))
    runs = []
    for s in range(2 * p):
        b, e = (int(min(max(o, 0), n)) for o in (offsets[s], offsets[s + 1]))
        runs.append((b, max(e, b)))
    share = np.array([beta / max(v[b:e].sum(), 1) if average else beta for b, e in runs])
    rewards = np.array([share[s] * d[b:e].sum() for s, (b, e) in enumerate(runs)])
    out = np.zeros(n) if dlogp is None else dlogp.copy()
    loss = 0.0
    for i in range(p):
        w = 1.0 / p if weight is None else weight[i]
        m = rewards[i] - rewards[p + i] - margin
        slope = 0.0
        if w != 0:
            loss += w * sum(f * _softplus(x) for f, x in ((1 - smoothing, -m), (smoothing, m)) if f)
            with np.errstate(over="ignore"):
                slope = dloss * w * (smoothing / (1 + np.exp(-m)) - (1 - smoothing) / (1 + np.exp(m)))
        for s, sign in ((i, 1.0), (p + i, -1.0)):
            b, e = runs[s]
            out[b:e] = np.where(v[b:e], sign * share[s] * slope, 0.0)
    return loss, rewards, out
