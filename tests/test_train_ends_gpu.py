"""The operators at the two ends of a training step together, as a loop uses
them: query and key heads normed and turned, attention (plain torch), a head
projection, the tokens' log-probabilities, a loss on them, the backward pass of
all of it, and the optimizer's steps on the gradients (muon_adamw_step on the
gains, muon_step on the weights).  Gradients are compared with those of the same
mathematics in fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import (AdamWGroup, MuonPlan, policy_loss, preference_loss, qk_norm_rope, qk_norm_rope_backward,
                                  token_logp, token_logp_backward)
from oracle import ends_ref as R
from tests.ops_helpers import DEV, draw

pytestmark = pytest.mark.gpu
B, T, C, HQ, HK, D, V, EPS, SCALE = 4, 24, 48, 4, 2, 16, 203, 1e-6, 0.9
LOW, HIGH, BETA = 0.2, 0.3, 0.05


def _setup():
    x = draw((B, T, C), 1)
    wqkv, wo, wv = draw(((HQ + 2 * HK) * D, C), 2, 0.2), draw((C, HQ * D), 3, 0.2), draw((V, C), 4, 0.3)
    gq, gk = draw((D,), 5, 0.1, 1.0), draw((D,), 6, 0.1, 1.0)
    rng = np.random.Generator(np.random.PCG64(7))
    targets = torch.from_numpy(rng.integers(0, V, (B, T)))
    targets[:, :3] = -100                                   # the prompt
    return [t.to(DEV) for t in (x, wqkv, wo, wv, gq, gk)], targets.to(DEV)


def _model64(x, wqkv, wo, wv, gq, gk, targets):
    """Log-probabilities in fp64, for automatic differentiation."""
    cn, sn = R.table(T, D)
    c, s = (torch.from_numpy(v.astype(np.float64)) for v in (cn, sn))
    qkv = (x @ wqkv.t()).view(B, T, HQ + 2 * HK, D)

    def head(h, g):
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * g
        a, b = y[..., :D // 2], y[..., D // 2:]
        c4, s4 = c[None, :, None], s[None, :, None]
        return torch.cat([a * c4 - b * s4, b * c4 + a * s4], -1)

    q, k, v = head(qkv[:, :, :HQ], gq), head(qkv[:, :, HQ:HQ + HK], gk), qkv[:, :, HQ + HK:]
    k, v = (t.repeat_interleave(HQ // HK, 2) for t in (k, v))
    a = torch.einsum("bihd,bjhd->bhij", q, k) / D ** 0.5
    a = a.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -torch.inf).softmax(-1)
    out = torch.einsum("bhij,bjhd->bihd", a, v).reshape(B, T, HQ * D)
    z = (x + out @ wo.t()) @ wv.t() * SCALE
    lp = torch.log_softmax(z, -1).gather(-1, targets.clamp(min=0)[..., None])[..., 0]
    return torch.where(targets >= 0, lp, torch.zeros(()).double())


def _forward(ws, targets, cos, sin):
    x, wqkv, wo, wv, gq, gk = ws
    qkv = (x @ wqkv.t()).view(B, T, HQ + 2 * HK, D)
    q, k, v = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:]
    qo = torch.empty(B, HQ, T, D, device=DEV).transpose(1, 2)
    ko = torch.empty(B, HK, T, D, device=DEV).transpose(1, 2)
    qk_norm_rope(q, k, gq, gk, cos, sin, qo, ko, eps=EPS)
    # attention and its backward pass are the caller's: torch in fp32 here
    leaves = [t.detach().clone().requires_grad_() for t in (qo, ko, v)]
    kk, vv = (t.repeat_interleave(HQ // HK, 2) for t in leaves[1:])
    qt, kt, vt = (t.transpose(1, 2).contiguous() for t in (leaves[0], kk, vv))
    a = torch.matmul(qt, kt.transpose(2, 3).contiguous()) / D ** 0.5
    a = a.masked_fill(torch.ones(T, T, dtype=torch.bool, device=DEV).triu(1), -torch.inf).softmax(-1)
    out = torch.matmul(a, vt).transpose(1, 2).reshape(B, T, HQ * D)
    hidden = x + out.detach() @ wo.t()
    logits = hidden @ wv.t()
    logp, lse = torch.empty(B, T, device=DEV), torch.empty(B, T, device=DEV)
    token_logp(logits, targets, logp, lse, scale=SCALE)
    return dict(qkv=qkv, q=q, k=k, leaves=leaves, out=out, hidden=hidden, logits=logits, logp=logp, lse=lse)


def _backward(ws, targets, cos, sin, f, dlogp, grads):
    x, wqkv, wo, wv, gq, gk = ws
    dlogits = f["logits"]                                    # in place: the logits are not needed again
    token_logp_backward(f["logits"], targets, f["logp"], f["lse"], dlogp, dlogits, scale=SCALE)
    d2 = dlogits.view(B * T, V)
    grads[2].copy_(d2.t().contiguous() @ f["hidden"].reshape(B * T, C))
    dhidden = d2 @ wv
    grads[1].copy_(dhidden.t().contiguous() @ f["out"].detach().reshape(B * T, HQ * D))
    dout = (dhidden @ wo).view(B, T, HQ * D)
    dqo, dko, dv = torch.autograd.grad(f["out"], f["leaves"], dout)
    dqkv = torch.empty_like(f["qkv"])
    qk_norm_rope_backward(dqo, dko, f["q"], f["k"], gq, gk, cos, sin, dqkv[:, :, :HQ], dqkv[:, :, HQ:HQ + HK],
                          dgamma_q=grads[3], dgamma_k=grads[4], eps=EPS)
    dqkv[:, :, HQ + HK:] = dv
    grads[0].copy_(dqkv.view(B * T, -1).t().contiguous() @ x.view(B * T, C))


def _loop(kind, steps):
    ws, targets = _setup()
    cn, sn = R.table(T, D)
    cos, sin = torch.from_numpy(cn).to(DEV), torch.from_numpy(sn).to(DEV)
    grads = [torch.empty_like(w) for w in ws[1:]]
    state = [torch.zeros_like(w) for w in ws[1:]] + [torch.zeros_like(w) for w in ws[4:]]
    plan = MuonPlan([w.shape for w in ws[1:4]], torch.float32)
    adam = AdamWGroup(ws[4:], grads[3:], state[3:5], state[5:])
    ref = _forward(ws, targets, cos, sin)["logp"].clone()
    old = ref + 0.1 * draw((B, T), 8).to(DEV)
    adv, w = draw((B, T), 9).to(DEV), (targets >= 0).float() / int((targets >= 0).sum())
    off = torch.arange(0, (B + 1) * T, T, device=DEV)
    log = []
    for step in range(steps):
        f = _forward(ws, targets, cos, sin)
        loss, dlogp = torch.empty(1, device=DEV), torch.empty_like(f["logp"])
        if kind == "policy":
            policy_loss(f["logp"], old, adv, loss, ref_logp=ref, weight=w, dlogp=dlogp, clip_low=LOW, clip_high=HIGH,
                        beta=BETA)
        else:
            preference_loss(f["logp"], off, loss, ref_logp=ref, valid=targets >= 0, dlogp=dlogp, beta=0.3)
        before = [p.clone() for p in ws]
        logp = f["logp"].clone()
        _backward(ws, targets, cos, sin, f, dlogp, grads)
        log.append(dict(ws=before, grads=[g.clone() for g in grads], loss=loss, logp=logp, old=old, ref=ref, adv=adv, w=w,
                        targets=targets))
        plan.step(ws[1:4], grads[:3], state[:3], lr=1e-2, wd=0.1)
        adam.step(lr=1e-2, wd=0.1, step=step + 1)
    torch.cuda.synchronize()
    return log


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_gradients_of_the_step(kind):
    for s in _loop(kind, 3):
        leaves = [t.double().cpu().requires_grad_() for t in s["ws"]]
        targets = s["targets"].cpu()
        lp = _model64(*leaves, targets)
        assert float((lp - s["logp"].double().cpu()).detach().abs().max()) < 1e-4
        old, ref, adv, w = (s[n].double().cpu() for n in ("old", "ref", "adv", "w"))
        if kind == "policy":
            ratio = torch.exp(lp - old)
            u = ref - lp
            pg = -torch.minimum(ratio * adv, ratio.clamp(1 - LOW, 1 + HIGH) * adv)
            f = (w * (pg + BETA * (torch.exp(u) - u - 1))).sum()
        else:
            r = 0.3 * torch.where(targets >= 0, lp - ref, torch.zeros(()).double()).sum(1)
            f = -torch.nn.functional.logsigmoid(r[:B // 2] - r[B // 2:]).mean()
        assert abs(float(s["loss"]) - float(f.detach())) < 1e-5
        want = torch.autograd.grad(f, leaves[1:])
        for name, g, v in zip(("wqkv", "wo", "wv", "gamma_q", "gamma_k"), s["grads"], want):
            # a chain of fp32 operators and products of length 203 at most: a few hundred roundings of 2^-24
            err = float((g.double().cpu() - v).norm() / v.norm())
            assert err < 1e-4, (name, err)


def test_the_loop_is_the_same_from_run_to_run():
    for a, b in zip(_loop("policy", 2), _loop("policy", 2)):
        assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["logp"], b["logp"])
        assert torch.equal(a["grads"][3], b["grads"][3]) and torch.equal(a["grads"][4], b["grads"][4])
