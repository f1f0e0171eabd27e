"""The training operators together, as a loop uses them beside the step: a
residual branch (dropout, add, norm), a router on the normalised tokens, a
linear mixture of its experts, the backward pass of all of it, and the
optimizer's steps on the gradients (muon_adamw_step on the gain and bias,
muon_step on the router and the expert slab).  Gradients are compared with
those of the same mathematics in fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import (AdamWGroup, MuonPlan, dropout_add_layer_norm, dropout_add_layer_norm_backward, route,
                                  route_backward)
from oracle import ops_ref as R
from tests.ops_helpers import DEV, draw

pytestmark = pytest.mark.gpu
T, C, E, KK, P, SEED, COEF, EPS = 96, 64, 8, 2, 0.1, 41, 0.02, 1e-5


def _forward64(x, res, gamma, beta, wr, we, keep, idx, counts, n):
    """Objective sum(out^2) / 2 + loss with the mask and the choices held."""
    h = res + torch.where(keep, x * (65536 / (65536 - R.threshold(P))), torch.zeros_like(x))
    mean = h.mean(1, keepdim=True)
    y = (h - mean) / torch.sqrt(((h - mean) ** 2).mean(1, keepdim=True) + EPS) * gamma + beta
    p = torch.softmax(y @ wr.t(), 1)
    q = p.gather(1, idx)
    gates = q / q.sum(1, keepdim=True)
    outs = torch.stack([y @ w for w in we], 1)                      # [T, E, C]
    out = h + (gates[..., None] * outs.gather(1, idx[..., None].expand(-1, -1, C))).sum(1)
    loss = COEF * E * (counts / (KK * n) * p.mean(0)).sum()
    return (out ** 2).sum() / 2 + loss


def _loop(steps, stream=None):
    x, res = draw((T, C), 1).to(DEV), draw((T, C), 2).to(DEV)
    gamma, beta = draw((C,), 3, 0.1, 1.0).to(DEV), draw((C,), 4, 0.1).to(DEV)
    wr, we = draw((E, C), 5, 0.3).to(DEV), draw((E, C, C), 6, 0.1).to(DEV)
    grads = [torch.empty_like(t) for t in (gamma, beta, wr, we)]
    moments = [torch.zeros_like(t) for t in (gamma, beta, gamma, beta, wr, we)]
    adam = AdamWGroup([gamma, beta], grads[:2], moments[:2], moments[2:4])
    plan = MuonPlan([wr.shape, we.shape], torch.float32)
    out = []
    for step in range(steps):
        h, y = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        rng = dict(p=P, seed=SEED, offset=step)
        dropout_add_layer_norm(x, res, gamma, beta, h, y, mean=mean, rstd=rstd, eps=EPS, **rng)
        logits = y @ wr.t()
        idx, gates = torch.empty(T, KK, dtype=torch.int32, device=DEV), torch.empty(T, KK, device=DEV)
        counts, n = torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
        loss = torch.empty(1, device=DEV)
        route(logits, idx, gates, counts, n, loss, coef=COEF)
        at = idx.long()
        outs = torch.stack([y @ w for w in we], 1)
        chosen = outs.gather(1, at[..., None].expand(-1, -1, C))
        full = h + (gates[..., None] * chosen).sum(1)
        before = [t.clone() for t in (gamma, beta, wr, we)]
        # backward
        dout = full
        dgates = (dout[:, None, :] * chosen).sum(2).contiguous()
        dlogits = torch.empty_like(logits)
        route_backward(logits, idx, counts, n, dlogits, dgates=dgates, coef=COEF)
        dy = dlogits @ wr
        for e in range(E):
            g = torch.where(at == e, gates, torch.zeros_like(gates)).sum(1, keepdim=True)
            dy += (g * dout) @ we[e].t().contiguous()
            grads[3][e] = y.t().contiguous() @ (g * dout)
        torch.mm(dlogits.t().contiguous(), y, out=grads[2])
        dx, dres = torch.empty_like(x), torch.empty_like(x)
        dropout_add_layer_norm_backward(dy, h, gamma, mean, rstd, dx, dres, dh=dout, dgamma=grads[0], dbeta=grads[1],
                                        **rng)
        out.append(dict(x=x, res=res, params=before, grads=[g.clone() for g in grads], dx=dx, dres=dres, idx=at,
                        counts=counts, n=n, loss=loss, step=step))
        adam.step(lr=1e-2, wd=0.1, step=step + 1)
        plan.step([wr, we], [grads[2], grads[3]], moments[4:], lr=1e-2, wd=0.1)
    torch.cuda.synchronize()
    return out


def test_gradients_of_the_block():
    for s in _loop(3):
        leaves = [t.double().cpu().requires_grad_() for t in (s["x"], s["res"], *s["params"])]
        keep = torch.from_numpy(R.keep_mask(T, C, P, SEED, s["step"]))
        f = _forward64(*leaves, keep, s["idx"].cpu(), s["counts"].double().cpu(), int(s["n"]))
        want = torch.autograd.grad(f, leaves)
        assert int(s["counts"].sum()) == T * KK and int(s["n"]) == T
        for name, g, w in zip(("dx", "dres", "dgamma", "dbeta", "drouter", "dexperts"),
                              (s["dx"], s["dres"], *s["grads"]), want):
            err = float((g.double().cpu() - w).norm() / w.norm())
            # a chain of fp32 operators and products of length 64: a few hundred roundings of 2^-24
            assert err < 1e-4, (name, err)


def test_the_loop_is_the_same_from_run_to_run():
    for a, b in zip(_loop(3), _loop(3)):
        for x, y in zip((a["dx"], a["dres"], a["loss"], *a["grads"]), (b["dx"], b["dres"], b["loss"], *b["grads"])):
            assert torch.equal(x, y)
