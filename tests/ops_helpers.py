"""Bounds and draws shared by the training operators' GPU tests.

Every bound is absolute and elementwise: half a step of the stored type on
the result (one rounding to nearest), plus the fp32 arithmetic before it.
That is counted in units u = 2^-24 (half a step of fp32) with the factor
K = 64: a sum over a row of up to 32768 elements is at most 32 additions in
a thread, 6 across a wave and 16 across waves, so its relative error (of the
sum of absolute values) is below 54 u, and the few products, divisions and
roots around it stay below 10 u more.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
K = 64
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def draw(shape, seed, std=1.0, mean=0.0, dtype=torch.float32):
    """A seeded host tensor rounded to dtype."""
    rng = np.random.Generator(np.random.PCG64(seed))
    return torch.from_numpy((rng.standard_normal(shape, dtype=np.float32) * np.float32(std) + np.float32(mean))).to(dtype)


def h64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def within(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, what: str):
    g = h64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    err = np.abs(g - want)
    bad = ~(err <= bound + 1e-37)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst "
                           f"{float(np.nanmax(err / (bound + 1e-37))):.2f}x")


def norm_bounds(x, gamma, beta, y, mean, rstd, dtype):
    """(y, mean, rstd) bounds of the forward pass; fp64 arrays."""
    a = np.abs(x).mean(1)
    d = np.abs(x - mean[:, None])
    # the deviations: their own rounding, and the mean's error
    dev = U * d + K * U * a[:, None]
    # rstd: half of the relative error of var + eps, whose sum of squares has the deviations' errors too
    rel = K * U + (2 * d * dev).mean(1) * rstd ** 2
    g = 1.0 if gamma is None else np.abs(gamma)
    b = 0.0 if beta is None else np.abs(beta)
    by = half_step(dtype) * np.abs(y) * (1 + 1e-6) + (dev + d * (rel[:, None] + 4 * U)) * rstd[:, None] * g * 1.01 \
        + 2 * U * (np.abs(y) + b)
    return by, K * U * a + U * np.abs(mean), rel * rstd + 4 * U * rstd


def norm_grad_bounds(dy, x, gamma, mean, rstd, dx, dtype, wdtype, rows_in_order):
    """(dx, dgamma, dbeta) bounds of the backward pass, given the same fp32
    mean and rstd; rows_in_order: the longest chain of additions over rows."""
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy if gamma is None else dy * gamma)
    inner = rstd[:, None] * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    chain = (rows_in_order + 64) * U
    bx = half_step(dtype) * np.abs(dx) * (1 + 1e-6) + K * U * inner
    sg, sb = (np.abs(dy) * xh).sum(0), np.abs(dy).sum(0)
    return bx, sg, sb, chain, half_step(wdtype)
