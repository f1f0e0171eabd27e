"""Cases of the operators at the two ends of a training step: the norm of every
query and key head with the position rotation, the log-probabilities of a
batch's tokens, and the clipped policy loss and the preference loss on them,
each direction.

With ``own`` false a pass computes the operator in elementary torch
operations in 32 bits (the losses' per-token terms and sums, a few numbers a
token, in 64: differences of log-probabilities next to 0 and to the clipping
border), rounded once per output; with ``own`` true it makes the calls of the
package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
NONE = -100  # a token without a target


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token's heads while sampling: launch latency
        dict(name="qk_fwd_one_token", op="qk_fwd", batch=1, seq=1, hq=32, hk=8, dim=128, rot=128, inter=False,
             layout="packed", pos=True, dt="bf16", wdt="bf16"),
        # a micro-batch of 4 x 4096 tokens at the mixed set's width (32 heads of 128), slices of the projection's output
        dict(name="qk_fwd_4x4096_packed", op="qk_fwd", batch=4, seq=4096, hq=32, hk=8, dim=128, rot=128, inter=False,
             layout="packed", pos=False, dt="bf16", wdt="bf16"),
        # fp32, odd token counts, half of each head turned, heads before tokens as attention takes them
        dict(name="qk_bwd_odd_f32", op="qk_bwd", batch=3, seq=613, hq=12, hk=4, dim=80, rot=40, inter=True,
             layout="heads", pos=True, dt="f32", wdt="f32"),
        # the large set's width (64 heads of 128), a long micro-batch, fp32 gains
        dict(name="qk_bwd_2x8192", op="qk_bwd", batch=2, seq=8192, hq=64, hk=8, dim=128, rot=128, inter=False,
             layout="packed", pos=False, dt="bf16", wdt="f32"),
        # one sampled token over a large vocabulary: latency, one row over the whole device
        dict(name="logp_fwd_one_row", op="logp_fwd", rows=1, vocab=131072, scale=1.0, ignored=0.0, pad=0, dt="bf16"),
        # the log-probabilities of a micro-batch
        dict(name="logp_fwd_8192x65536", op="logp_fwd", rows=8192, vocab=65536, scale=1.0, ignored=0.0, pad=0, dt="bf16"),
        # fp32 logits of odd width with padding tokens, sampled at a temperature
        dict(name="logp_bwd_odd_f32", op="logp_bwd", rows=515, vocab=50021, scale=1.25, ignored=0.3, pad=11, dt="f32"),
        # their gradient for the micro-batch, prompt tokens without a target
        dict(name="logp_bwd_8192x65536", op="logp_bwd", rows=8192, vocab=65536, scale=1.0, ignored=0.1, pad=0, dt="bf16"),
        # a small batch of sampled answers: latency
        dict(name="policy_777", op="policy", rows=777, ref=False, old=True, weights=True, beta=0.0),
        # a large one with a reference model
        dict(name="policy_262144", op="policy", rows=262144, ref=True, old=True, weights=True, beta=0.04),
        # four short pairs of answers
        dict(name="preference_4_pairs", op="pref", pairs=4, mean=300, ref=True, weights=False, average=False, beta=0.1,
             margin=0.0, smoothing=0.0),
        # many long ones, means instead of sums
        dict(name="preference_96_pairs", op="pref", pairs=96, mean=4096, ref=True, weights=True, average=True, beta=2.0,
             margin=0.5, smoothing=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "logp_fwd", "logp_bwd", "policy", "pref"])
    dt = rng.choice(["bf16", "f32"])
    if op.startswith("qk"):
        dim = rng.choice([32, 64, 80, 96, 112, 128, 160, 192, 256, 2 * rng.randint(8, 128)])
        rot = rng.choice([dim, dim, dim // 2 // 2 * 2, 2 * rng.randint(1, dim // 2)])
        hk = rng.randint(1, 12)
        hq = hk * rng.randint(1, 8)
        tokens = _log(rng, 1, min(32768, (1 << 26) // ((hq + hk) * dim)))
        batch = rng.randint(1, min(8, tokens))
        return dict(op=op, batch=batch, seq=max(tokens // batch, 1), hq=hq, hk=hk, dim=dim, rot=rot,
                    inter=rng.random() < 0.4, layout=rng.choice(["packed", "plain", "heads"]),
                    pos=rng.random() < 0.5, dt=dt, wdt=rng.choice(["bf16", "f32"]))
    if op.startswith("logp"):
        vocab = _log(rng, 100, 262144)
        if rng.random() < 0.5:
            vocab = (vocab + 63) // 64 * 64
        return dict(op=op, rows=_log(rng, 1, min(32768, (1 << 28) // vocab)), vocab=vocab,
                    scale=rng.choice([1.0, 1.0, 0.7, 1.25]), ignored=rng.choice([0.0, 0.1, 0.5]),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), dt=dt)
    if op == "policy":
        ref = rng.random() < 0.6
        return dict(op=op, rows=_log(rng, 1, 1 << 20), ref=ref, old=rng.random() < 0.8, weights=rng.random() < 0.8,
                    beta=rng.choice([0.01, 0.04, 0.2]) if ref else 0.0)
    mean = _log(rng, 1, 16384)
    average = rng.random() < 0.4
    return dict(op=op, pairs=_log(rng, 1, min(512, (1 << 20) // mean)), mean=mean, ref=rng.random() < 0.7,
                weights=rng.random() < 0.5, average=average, beta=2.0 if average else rng.choice([0.05, 0.1]),
                margin=rng.choice([0.0, 0.5]), smoothing=rng.choice([0.0, 0.1]))


def work(case):
    op = case["op"]
    if op.startswith("qk"):
        t, b, w = case["batch"] * case["seq"], SIZE[case["dt"]], SIZE[case["wdt"]]
        n = t * (case["hq"] + case["hk"]) * case["dim"]
        # angles are read once for each position
        angles = 4 * case["rot"] * (t if case["pos"] else case["seq"]) + (8 * t if case["pos"] else 0)
        if op == "qk_fwd":
            return {"bytes": 2 * n * b + 2 * case["dim"] * w + angles, "flops": 8 * n}
        return {"bytes": 3 * n * b + 4 * case["dim"] * w + angles, "flops": 16 * n}
    if op.startswith("logp"):
        n, r = case["rows"] * case["vocab"], case["rows"]
        live = max(1, round(r * (1 - case["ignored"])))
        read = live * case["vocab"] * SIZE[case["dt"]]  # a token without a target has no logits to read
        if op == "logp_fwd":
            return {"bytes": read + 16 * r, "flops": 5 * live * case["vocab"]}
        return {"bytes": read + n * SIZE[case["dt"]] + 20 * r, "flops": 5 * live * case["vocab"]}
    if op == "policy":
        arrays = 3 + case["ref"] + case["old"] + case["weights"]
        return {"bytes": 4 * arrays * case["rows"] + 16, "flops": 20 * case["rows"]}
    tokens = 2 * case["pairs"] * case["mean"]
    return {"bytes": 4 * (2 + case["ref"]) * tokens + 40 * case["pairs"], "flops": 3 * tokens}


# ---- inputs ------------------------------------------------------------------

def _heads(case, heads, dt, packed=None):
    """Empty [batch, seq, heads, dim] in the case's layout; `packed` is the
    buffer [batch, seq, all heads, dim] and the first head of a slice."""
    b, s, d = case["batch"], case["seq"], case["dim"]
    if case["layout"] == "packed":
        buf, first = packed
        return buf[:, :, first:first + heads]
    if case["layout"] == "heads":
        return torch.empty((b, heads, s, d), dtype=dt, device=DEV).transpose(1, 2)
    return torch.empty((b, s, heads, d), dtype=dt, device=DEV)


def _pair(case, dt):
    """Queries' and keys' tensors, slices of one buffer (with values behind them) if packed."""
    hq, hk = case["hq"], case["hk"]
    buf = None
    if case["layout"] == "packed":
        buf = torch.empty((case["batch"], case["seq"], hq + 2 * hk, case["dim"]), dtype=dt, device=DEV)
    return _heads(case, hq, dt, (buf, 0)), _heads(case, hk, dt, (buf, hq))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}

    def normal(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean)

    if op.startswith("qk"):
        dt, wdt, dim = DT[case["dt"]], DT[case["wdt"]], case["dim"]
        b, n = case["batch"], case["seq"]
        table = 4 * n + 5
        # sharp to flat heads: their lengths differ by a factor of about ten
        for name, t in zip("qk", _pair(case, dt)):
            t.copy_(normal(t.shape) * torch.exp(normal((1, 1, t.shape[2], 1), 0.6)))
            s[name] = t
        s["gq"], s["gk"] = normal(dim, 0.2, 1.0).to(wdt), normal(dim, 0.2, 1.0).to(wdt)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / max(case["rot"], 1))
        angle = torch.arange(table, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        s["pos"] = None
        if case["pos"]:  # each sequence starts somewhere else in its document
            first = torch.randint(0, table - n, (b, 1), generator=g, device=DEV)
            s["pos"] = (first + torch.arange(n, device=DEV)).contiguous()
        s["qo"], s["ko"] = _pair(case, dt) if op == "qk_bwd" else (_heads(dict(case, layout="heads"), case["hq"], dt),
                                                                  _heads(dict(case, layout="heads"), case["hk"], dt))
        if op == "qk_bwd":
            for name, h in (("dq", case["hq"]), ("dk", case["hk"])):  # what attention's backward pass gives
                t = _heads(dict(case, layout="heads"), h, dt)
                t.copy_(normal(t.shape, 1e-2))
                s[name] = t
            s["dgq"], s["dgk"] = torch.empty_like(s["gq"]), torch.empty_like(s["gk"])
        return s
    if op.startswith("logp"):
        r, v, dt = case["rows"], case["vocab"], DT[case["dt"]]
        x = torch.empty((r, v + case["pad"]), dtype=dt, device=DEV)[:, :v]
        for i in range(0, r, 1024):
            x[i:i + 1024] = normal((min(1024, r - i), v), 2.0)
        t = torch.randint(0, v, (r,), generator=g, device=DEV)
        # most tokens are likely ones: their logits stand above the others by up to 20
        lift = torch.rand(r, generator=g, device=DEV) * 20
        x.scatter_(1, t[:, None], (x.gather(1, t[:, None]).float() + lift[:, None]).to(dt))
        if case["ignored"]:
            t[torch.rand(r, generator=g, device=DEV) < case["ignored"]] = NONE
        s.update(logits=x, targets=t, logp=torch.empty(r, device=DEV), lse=torch.empty(r, device=DEV))
        if op == "logp_bwd":
            logp, lse = _exact_logp(s, case)
            s["logp"], s["lse"] = logp.float(), lse.float()
            s["dlogp"] = normal(r, 1e-3)
            s["dlogits"] = torch.empty((r, v + case["pad"]), dtype=dt, device=DEV)[:, :v]
        return s
    if op == "policy":
        r = case["rows"]
        s["logp"] = -torch.exp(normal(r, 2.0, -1.5))
        s["old"] = (s["logp"] + normal(r, 0.15)).clamp(max=0) if case["old"] else None
        s["ref"] = (s["logp"] + normal(r, 0.3)).clamp(max=0) if case["ref"] else None
        s["adv"] = normal(r)
        s["w"] = None
        if case["weights"]:  # prompt and padding tokens count nothing, the others alike
            keep = torch.rand(r, generator=g, device=DEV) < 0.8
            s["w"] = keep.float() / keep.sum().clamp(min=1)
        s.update(loss=torch.empty(1, device=DEV), terms=torch.empty(3, device=DEV), dlogp=torch.empty(r, device=DEV))
        return s
    p = case["pairs"]
    n = 2 * p * case["mean"]  # cut anywhere: answers from empty ones to several times the mean
    cuts = torch.randint(0, n + 1, (2 * p + 1,), generator=g, device=DEV).sort().values
    cuts[0], cuts[-1] = 0, n
    s["offsets"] = cuts
    s["logp"] = -torch.exp(normal(n, 2.0, -1.5))
    s["ref"] = (s["logp"] + normal(n, 0.1)).clamp(max=0) if case["ref"] else None
    s["w"] = torch.rand(p, generator=g, device=DEV) / p if case["weights"] else None
    s.update(loss=torch.empty(1, device=DEV), rewards=torch.empty(2 * p, device=DEV), dlogp=torch.empty(n, device=DEV))
    return s


# ---- plain forms ---------------------------------------------------------------

def _angles(s):
    """cos and sin of every token, [batch or 1, seq, 1, rot / 2]."""
    if s["pos"] is None:
        n = s["case"]["seq"]
        return s["cos"][None, :n, None], s["sin"][None, :n, None]
    return s["cos"][s["pos"]][:, :, None], s["sin"][s["pos"]][:, :, None]


def _turn(y, cos, sin, rot, inter):
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., rot:]], -1)
    h = rot // 2
    a, b = y[..., :h], y[..., h:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)


def _qk_plain(s, x, gamma, dt):
    case = s["case"]
    cos, sin = _angles(s)
    x = x.float()
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
    return _turn(x * r * gamma.float(), cos, sin, case["rot"], case["inter"]).to(dt)


def _qk_grad_plain(s, dy, x, gamma, dt):
    case = s["case"]
    cos, sin = _angles(s)
    x, gm = x.float(), gamma.float()
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
    g = _turn(dy.float(), cos, -sin, case["rot"], case["inter"])
    dgamma = (g * (x * r)).flatten(0, 2).sum(0)
    g = g * gm
    dx = r * (g - x * (r * r * ((g * x).sum(-1, keepdim=True) / case["dim"])))
    return dx.to(dt), dgamma.to(gamma.dtype)


def _logp_plain(s, case):
    z, t = s["logits"].float() * case["scale"], s["targets"]
    some = t >= 0
    at = t.clamp(min=0)[:, None]
    top = z.max(1, keepdim=True).values
    zt = z.gather(1, at) - top
    # the target apart from the others: where it is nearly certain its logarithm is that of a sum next to 1
    rest = torch.exp(z - top).scatter_(1, at, 0.0).sum(1, keepdim=True)
    et = torch.exp(zt)
    ratio = rest / et
    logp = torch.where(ratio < 1, -torch.log1p(ratio), zt - torch.log(et + rest))
    lse = top + torch.log(et + rest)
    zero = torch.zeros((), device=DEV)
    return torch.where(some, logp[:, 0], zero), torch.where(some, lse[:, 0], zero)


def _logp_grad_plain(s, case):
    t = s["targets"]
    some = (t >= 0)[:, None]
    at = t.clamp(min=0)[:, None]
    p = torch.exp(s["logits"].float() * case["scale"] - s["lse"][:, None])
    d = (-p).scatter_(1, at, -torch.expm1(s["logp"])[:, None])
    d = d * (s["dlogp"][:, None] * case["scale"])
    return torch.where(some, d, torch.zeros((), device=DEV)).to(s["logits"].dtype)


LOW, HIGH = 0.2, 0.28


def _policy_plain(s, case):
    lp, adv = s["logp"].double(), s["adv"].double()
    d = lp - (lp if s["old"] is None else s["old"].double())
    ratio = torch.exp(d)
    low, high = 1 - float(np.float32(LOW)), 1 + float(np.float32(HIGH))
    cut = ((adv > 0) & (d > math.log(high))) | ((adv < 0) & (d < math.log(low)))
    border = low + (high - low) * (adv > 0).double()
    pg = -adv * torch.where(cut, border, ratio)
    dpg = torch.where(cut, torch.zeros_like(adv), -adv * ratio)
    beta = float(np.float32(case["beta"]))
    kl, dkl = torch.zeros_like(lp), torch.zeros_like(lp)
    if s["ref"] is not None:
        u = s["ref"].double() - lp
        kl, dkl = torch.expm1(u) - u, -torch.expm1(u)
    w = torch.ones_like(lp) if s["w"] is None else s["w"].double()
    terms = torch.stack([(w * pg).sum(), (w * kl).sum(), (w * cut).sum()])
    loss = terms[0] + beta * terms[1]
    return loss.float().reshape(1), terms.float(), (w * (dpg + beta * dkl)).float()


def _pref_plain(s, case):
    p = case["pairs"]
    d = s["logp"].double()
    if s["ref"] is not None:
        d = d - s["ref"].double()
    off = s["offsets"]
    lens = off[1:] - off[:-1]
    which = torch.repeat_interleave(torch.arange(2 * p, device=DEV), lens, output_size=d.numel())
    total = torch.zeros(2 * p, dtype=torch.float64, device=DEV).index_add_(0, which, d)
    share = 1 / lens.clamp(min=1).double() if case["average"] else torch.ones_like(total)
    beta, margin, ls = (float(np.float32(case[k])) for k in ("beta", "margin", "smoothing"))
    rewards = beta * share * total
    h = rewards[:p] - rewards[p:] - margin
    w = torch.full_like(h, 1 / p) if s["w"] is None else s["w"].double()
    wins = torch.log1p(torch.exp(-h.abs())) + (-h).clamp(min=0)  # -log sigmoid(h)
    loses = torch.log1p(torch.exp(-h.abs())) + h.clamp(min=0)
    loss = (w * ((1 - ls) * wins + ls * loses)).sum()
    dh = w * (ls - 1 / (1 + torch.exp(h)))
    each = beta * share * torch.cat([dh, -dh])
    return loss.float().reshape(1), rewards.float(), each[which].float()


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "policy":
        return _policy_plain(s, case)
    if op == "pref":
        return _pref_plain(s, case)
    if op == "logp_fwd":
        return _logp_plain(s, case)
    if op == "logp_bwd":
        return _logp_grad_plain(s, case)
    dt = DT[case["dt"]]
    if op == "qk_fwd":
        return [_qk_plain(s, s["q"], s["gq"], dt), _qk_plain(s, s["k"], s["gk"], dt)]
    dq, dgq = _qk_grad_plain(s, s["dq"], s["q"], s["gq"], dt)
    dk, dgk = _qk_grad_plain(s, s["dk"], s["k"], s["gk"], dt)
    return [dq, dk, dgq, dgk]


# ---- a pass ------------------------------------------------------------------------

def run(s):
    if not own:
        return _run_plain(s)
    import newton_schulz_05_amd as muon

    case = s["case"]
    op = case["op"]
    if op == "qk_fwd":
        muon.qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"], s["qo"], s["ko"], positions=s["pos"],
                          interleaved=case["inter"], eps=EPS)
        return [s["qo"], s["ko"]]
    if op == "qk_bwd":
        muon.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"], s["qo"],
                                   s["ko"], dgamma_q=s["dgq"], dgamma_k=s["dgk"], positions=s["pos"],
                                   interleaved=case["inter"], eps=EPS)
        return [s["qo"], s["ko"], s["dgq"], s["dgk"]]
    if op == "logp_fwd":
        muon.token_logp(s["logits"], s["targets"], s["logp"], s["lse"], scale=case["scale"])
        return s["logp"], s["lse"]
    if op == "logp_bwd":
        muon.token_logp_backward(s["logits"], s["targets"], s["logp"], s["lse"], s["dlogp"], s["dlogits"],
                                 scale=case["scale"])
        return s["dlogits"]
    if op == "policy":
        muon.policy_loss(s["logp"], s["old"], s["adv"], s["loss"], ref_logp=s["ref"], weight=s["w"], dlogp=s["dlogp"],
                         terms=s["terms"], clip_low=LOW, clip_high=HIGH, beta=case["beta"])
        return s["loss"], s["terms"], s["dlogp"]
    muon.preference_loss(s["logp"], s["offsets"], s["loss"], ref_logp=s["ref"], weight=s["w"], rewards=s["rewards"],
                         dlogp=s["dlogp"], beta=case["beta"], margin=case["margin"], smoothing=case["smoothing"],
                         average=case["average"])
    return s["loss"], s["rewards"], s["dlogp"]


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_logp(s, case):
    """(logp, lse) of the definition, some rows at a time; 0 without a target."""
    logits, t = s["logits"], s["targets"]
    logp = torch.zeros(case["rows"], dtype=torch.float64, device=DEV)
    lse = torch.zeros_like(logp)
    step = max(1, (1 << 26) // case["vocab"])
    for i in range(0, case["rows"], step):
        z = logits[i:i + step].double() * float(np.float32(case["scale"]))
        at = t[i:i + step]
        l = torch.logsumexp(z, 1)
        own_z = z.gather(1, at.clamp(min=0)[:, None])[:, 0]
        # log p = -log(1 + sum of the others over the target's own)
        others = torch.logsumexp(z.scatter(1, at.clamp(min=0)[:, None], -math.inf), 1) - own_z
        exact = -torch.logaddexp(others, torch.zeros_like(others))
        exact = torch.where(others < 0, -torch.log1p(torch.exp(others)), exact)
        logp[i:i + step] = torch.where(at >= 0, exact, 0.0)
        lse[i:i + step] = torch.where(at >= 0, l, 0.0)
    return logp, lse


def _rotation(s, x, back):
    """x as complex pairs times exp(+- i angle)."""
    case = s["case"]
    rot, t = case["rot"], x.clone()
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    turn = turn[:case["seq"]].unsqueeze(0) if s["pos"] is None else turn[s["pos"].reshape(-1)].reshape(*s["pos"].shape, -1)
    turn = (turn.conj() if back else turn).unsqueeze(2)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., one], x[..., two]) * turn
    t[..., one], t[..., two] = z.real, z.imag
    return t


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "logp_fwd":
        return _exact_logp(s, case)
    if op == "logp_bwd":
        out = torch.zeros((case["rows"], case["vocab"]), dtype=torch.float64, device=DEV)
        scale = float(np.float32(case["scale"]))
        rows = torch.nonzero(s["targets"] >= 0)[:, 0]
        step = max(1, (1 << 26) // case["vocab"])
        for i in range(0, rows.numel(), step):
            r = rows[i:i + step]
            p = torch.exp(s["logits"][r].double() * scale - s["lse"][r].double()[:, None])
            hit = torch.arange(len(r), device=DEV), s["targets"][r]
            p[hit] = torch.expm1(s["logp"][r].double())
            out[r] = p * (-scale * s["dlogp"][r].double()[:, None])
        return out
    if op.startswith("qk"):
        outs, grads = [], []
        for x, gm, dy in ((s["q"], s["gq"], s.get("dq")), (s["k"], s["gk"], s.get("dk"))):
            x, gm = x.double(), gm.double()
            unit = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
            if op == "qk_fwd":
                outs.append(_rotation(s, unit * gm, False))
                continue
            g = _rotation(s, dy.double(), True)
            grads.append((g * unit).sum((0, 1, 2)))
            g = g * gm
            outs.append((g - unit * (g * unit).mean(-1, keepdim=True)) * (x.square().mean(-1, keepdim=True) + EPS).rsqrt())
        return outs + grads
    f32 = lambda v: float(np.float32(v))  # noqa: E731 - a parameter as the call takes it
    lp = s["logp"].cpu().numpy().astype(np.float64)
    ref = None if s["ref"] is None else s["ref"].cpu().numpy().astype(np.float64)
    w = None if s["w"] is None else s["w"].cpu().numpy().astype(np.float64)
    if op == "policy":
        adv = s["adv"].cpu().numpy().astype(np.float64)
        gap = np.zeros_like(lp) if s["old"] is None else lp - s["old"].cpu().numpy().astype(np.float64)
        if w is None:
            w = np.ones_like(lp)
        hi, lo = 1 + f32(HIGH), 1 - f32(LOW)
        out = np.where(adv > 0, gap > np.log(hi), (adv < 0) & (gap < np.log(lo)))
        gain = np.minimum(np.exp(gap) * adv, np.clip(np.exp(gap), lo, hi) * adv)
        slope = np.where(out, 0.0, np.exp(gap) * adv)
        kl, pull = np.zeros_like(lp), np.zeros_like(lp)
        if ref is not None:
            kl, pull = np.expm1(ref - lp) - (ref - lp), np.expm1(ref - lp)
        a, b, c = math.fsum(-w * gain), math.fsum(w * kl), math.fsum(w * out)
        res = ([a + f32(case["beta"]) * b], [a, b, c], -w * (slope + f32(case["beta"]) * pull))
    else:
        p = case["pairs"]
        off = s["offsets"].cpu().numpy()
        ratio = lp if ref is None else lp - ref
        scale = np.array([f32(case["beta"]) / (max(off[i + 1] - off[i], 1) if case["average"] else 1) for i in range(2 * p)])
        rewards = scale * [math.fsum(ratio[off[i]:off[i + 1]]) for i in range(2 * p)]
        h = rewards[:p] - rewards[p:] - f32(case["margin"])
        ls = f32(case["smoothing"])
        w = np.full(p, 1 / p) if w is None else w
        loss = math.fsum(w * ((1 - ls) * np.logaddexp(0, -h) + ls * np.logaddexp(0, h)))
        up = w * (ls * 0.5 * (1 + np.tanh(h / 2)) - (1 - ls) * 0.5 * (1 - np.tanh(h / 2)))
        grad = np.zeros_like(lp)
        for i in range(p):
            grad[off[i]:off[i + 1]] = up[i] * scale[i]
            grad[off[p + i]:off[p + i + 1]] = -up[i] * scale[p + i]
        res = ([loss], rewards, grad)
    return tuple(torch.tensor(np.asarray(v), dtype=torch.float64, device=DEV) for v in res)
