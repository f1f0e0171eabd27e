"""Plain fp64 CPU oracle for the training operators beside the step: layer
norm, dropout, their fusion with the residual add, and the expert router.

TEST INFRASTRUCTURE ONLY, like muon_ref: only the test suite may import it,
and it imports nothing from the product path.  The formulas are those that
include/muon.h states; every operation is a fp64 NumPy expression (integers
for the generator and the choices).
"""
from __future__ import annotations

import numpy as np

M32 = np.uint64(0xFFFFFFFF)


# ---- layer norm ----------------------------------------------------------------

def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of x [rows, cols]; gamma / beta may be None."""
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta)."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---- dropout --------------------------------------------------------------------

def philox(counter, key, rounds=10):
    """Philox4x32 of uint64 arrays holding 32-bit words: counter (4), key (2)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [np.uint64(v) for v in key]
    for _ in range(rounds):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & M32, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + np.uint64(0x9E3779B9)) & M32, (k[1] + np.uint64(0xBB67AE85)) & M32]
    return c


def threshold(p):
    """Draws below this are dropped: p to the nearest 2^-16 (p taken in fp32)."""
    return int(np.rint(float(np.float32(p)) * 65536))


def keep_mask(rows, cols, p, seed, offset, first_row=0):
    """Kept elements (bool) of rows first_row .. first_row + rows - 1."""
    nb = -(-cols // 8)
    block, row = np.meshgrid(np.arange(nb, dtype=np.uint64), np.arange(first_row, first_row + rows, dtype=np.uint64))
    offset %= 1 << 64
    w = philox([block, row, np.uint64(offset & 0xFFFFFFFF), np.uint64(offset >> 32)],
               [seed & 0xFFFFFFFF, seed >> 32])
    u = np.stack([np.stack([v & np.uint64(0xFFFF), v >> np.uint64(16)], -1) for v in
                  (np.broadcast_to(x, block.shape) for x in w)], -2)
    return u.reshape(rows, nb * 8)[:, :cols] >= threshold(p)


def dropout(x, p, seed, offset, residual=None):
    t = threshold(p)
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    with np.errstate(invalid="ignore"):
        y = np.where(keep_mask(*x.shape, p, seed, offset), x * scale, 0.0)
    return y if residual is None else residual + y


# ---- router --------------------------------------------------------------------

def softmax_rows(x, valid=None):
    """(p, live): p is 0 in rows without a finite logit or not valid."""
    live = np.isfinite(x).any(1)
    if valid is not None:
        live = live & (np.asarray(valid) != 0)
    top = np.where(live, np.where(np.isfinite(x), x, -np.inf).max(1, initial=-np.inf), 0.0)
    with np.errstate(invalid="ignore"):
        z = np.where(live[:, None] & (x > -np.inf), np.exp(x - top[:, None]), 0.0)
    return z / np.where(live, z.sum(1), 1.0)[:, None], live


def route(x, k, coef, renorm, valid=None):
    """(indices, gates, counts, n, prob_mean, loss) of logits x [tokens, experts]."""
    p, live = softmax_rows(x, valid)
    e = x.shape[1]
    masked = np.where(live[:, None], x, -np.inf)
    order = np.argsort(-masked, axis=1, kind="stable")[:, :k]
    good = np.take_along_axis(masked, order, 1) > -np.inf
    gates = np.where(good, np.take_along_axis(p, order, 1), 0.0)
    if renorm:
        gates = gates / np.where(live, gates.sum(1), 1.0)[:, None]
    counts = np.bincount(order[good], minlength=e)
    n = int(live.sum())
    mean = p.sum(0) / max(n, 1)
    loss = coef * e * (counts / (k * max(n, 1)) * mean).sum()
    return np.where(good, order, -1), gates, counts, n, mean, loss


def route_objective(x, idx, counts, n, k, coef, renorm, dgates, dloss, valid=None):
    """sum(dgates * gates) + dloss * loss with the choices and counts held: what
    route_backward is the gradient of."""
    p, live = softmax_rows(x, valid)
    loss = coef * x.shape[1] * (counts / (k * max(n, 1)) * (p.sum(0) / max(n, 1))).sum()
    q = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0), 1), 0.0)
    if renorm:
        q = q / np.where(live, q.sum(1), 1.0)[:, None]
    return (dgates * q).sum() + dloss * loss


def route_backward(x, idx, counts, n, k, coef, renorm, dgates, dloss, valid=None):
    p, live = softmax_rows(x, valid)
    rows, e = x.shape
    dp = np.broadcast_to(dloss * coef * e * np.asarray(counts, float) / (k * max(n, 1) ** 2), (rows, e)).copy()
    good = idx >= 0
    at = np.maximum(idx, 0)
    dg = np.where(good, dgates, 0.0)
    if renorm:
        q = np.where(good, np.take_along_axis(p, at, 1), 0.0)
        s = np.where(q.sum(1) > 0, q.sum(1), 1.0)[:, None]  # without a choice there is no gradient
        dg = np.where(good, (dg - (dg * q).sum(1, keepdims=True) / s) / s, 0.0)
    for j in range(idx.shape[1]):
        np.add.at(dp, (np.arange(rows), at[:, j]), dg[:, j])
    return p * (dp - (p * dp).sum(1, keepdims=True))
