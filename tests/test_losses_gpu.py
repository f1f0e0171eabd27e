"""GPU policy loss and preference loss, with their gradients, against the fp64
oracle.  Everything is formed in fp64: results are off by one rounding to fp32
and by fp64 roundings, counted generously as 1e-12 of the sum of magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import MuonError, policy_loss, preference_loss
from oracle import ends_ref as R
from tests.ops_helpers import DEV, U, draw, h64, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
f32 = lambda v: float(np.float32(v))


def _opt(a):
    return None if a is None else h64(a)


def _one(got, want, scale, what):
    within(got, np.atleast_1d(np.asarray(want, float)), np.atleast_1d(U * np.abs(want) * 1.01 + 1e-12 * scale), what)


def _policy_inputs(n, seed, old=True, ref=True, weighted=True):
    lp = -torch.exp(draw((n,), seed, 2.0, -1.0)).to(DEV)
    ol = lp + draw((n,), seed + 1, 0.2).to(DEV) if old else None
    rf = lp + draw((n,), seed + 2, 0.3).to(DEV) if ref else None
    adv = draw((n,), seed + 3).to(DEV)
    w = None
    if weighted:
        keep = draw((n,), seed + 4).to(DEV) > -0.8
        w = keep.float() / max(int(keep.sum()), 1)
    return lp, ol, rf, adv, w


def _policy(lp, ol, rf, adv, w, low=0.2, high=0.28, beta=0.1, dloss=None, **kw):
    loss, terms, g = torch.full((1,), 7.0, device=DEV), torch.full((3,), 7.0, device=DEV), torch.full_like(lp, 7.0)
    policy_loss(lp, ol, adv, loss, ref_logp=rf, weight=w, dlogp=g, dloss=dloss, terms=terms, clip_low=low, clip_high=high,
                beta=beta, **kw)
    return loss, terms, g


def _check_policy(lp, ol, rf, adv, w, out, low=0.2, high=0.28, beta=0.1, dloss=1.0):
    want, terms, g = R.policy_loss(h64(lp), _opt(ol), _opt(rf), h64(adv), _opt(w), f32(low), f32(high), f32(beta), f32(dloss))
    size = np.abs(g).sum() + np.abs(terms).sum() + 1
    _one(out[0], want, size, "loss")
    _one(out[1], np.array(terms), size, "terms")
    _one(out[2], g, np.abs(g) + 1e-3, "dlogp")


@pytest.mark.parametrize("n", [1, 2, 63, 777, 1024, 1025, 4096, 4097, 5000, 60001, 300000])
@pytest.mark.parametrize("old,ref,weighted", [(True, True, True), (True, False, False), (False, True, True)])
def test_policy(n, old, ref, weighted):
    a = _policy_inputs(n, n, old, ref, weighted)
    out = _policy(*a)
    _check_policy(*a, out)
    again = _policy(*a, workspace=torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device=DEV))
    assert all(torch.equal(x, y) for x, y in zip(out, again))


def test_policy_scalars_and_optional_outputs():
    a = _policy_inputs(3000, 5)
    for low, high, beta, dl in ((0.0, 0.0, 0.0, None), (1.0, 3.0, -0.5, 2.5), (0.2, 0.2, 0.01, -1.0), (0.1, 0.0, 0.3, 0.0)):
        up = None if dl is None else torch.tensor([dl], device=DEV)
        out = _policy(*a, low=low, high=high, beta=beta, dloss=up)
        _check_policy(*a, out, low=low, high=high, beta=beta, dloss=1.0 if dl is None else dl)
        loss = torch.empty(1, device=DEV)
        policy_loss(a[0], a[1], a[3], loss, ref_logp=a[2], weight=a[4], clip_low=low, clip_high=high, beta=beta)
        assert torch.equal(loss, out[0])


def test_policy_next_to_the_border_and_to_zero():
    """Tokens within a few fp32 steps of the clipping border fall on its right
    side; the KL term of nearly equal policies keeps its relative accuracy."""
    n = 4000
    base = -torch.linspace(0.01, 6, n, device=DEV)
    edge = np.where(np.arange(n) % 2, np.log1p(0.25), np.log1p(-0.25))
    old = (base.double() - torch.from_numpy(edge).to(DEV)).float()
    old = old + (torch.arange(n, device=DEV) % 5 - 2) * 2 ** -22 * old.abs()
    adv = torch.where(torch.arange(n, device=DEV) % 3 == 0, -1.0, 1.0)
    ref = base * (1 + 1e-6 * draw((n,), 8).to(DEV))
    out = _policy(base, old, ref, adv, None, low=0.25, high=0.25, beta=1e6)
    _check_policy(base, old, ref, adv, None, out, low=0.25, high=0.25, beta=1e6)
    kl = R.policy_loss(h64(base), None, h64(ref), np.zeros(n), None, 0.2, 0.2, 1.0)[1][1]
    same = _policy(base, None, ref, torch.zeros(n, device=DEV), None, beta=1.0)
    assert 0 < kl < 1e-6 and abs(float(same[1][1]) - kl) < 1e-6 * kl
    # equal policies: ratio 1, no KL, gradient -A
    out = _policy(base, base.clone(), base.clone(), adv, None)
    assert out[1][1] == 0 and out[1][2] == 0 and torch.equal(out[2], -adv)


def test_policy_tokens_that_do_not_count():
    n = 9000
    lp, ol, rf, adv, w = _policy_inputs(n, 9)
    want = _policy(lp, ol, rf, adv, w)
    off = w == 0
    assert off.any()
    for t, v in ((lp, NAN), (ol, INF), (rf, -INF), (adv, NAN)):
        t[off] = v
    got = _policy(lp, ol, rf, adv, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[2][off].any()
    none = _policy(lp, ol, rf, adv, torch.zeros(n, device=DEV))
    assert not none[0].any() and not none[1].any() and not none[2].any()
    # what a counted token holds shows
    lp[0], w[0] = NAN, 0.5
    bad = _policy(lp, ol, rf, adv, w)
    assert torch.isnan(bad[0]).all() and torch.isnan(bad[2][0]) and torch.equal(bad[2][1:], want[2][1:])


def test_policy_extreme_ratios():
    lp = torch.tensor([0.0, 0.0, -1000.0, -1000.0, 0.0, -INF, -INF], device=DEV)
    ol = torch.tensor([-1000.0, -1000.0, 0.0, 0.0, -1000.0, -1.0, -1.0], device=DEV)
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 0.0, 1.0, -1.0], device=DEV)
    out = _policy(lp, ol, None, adv, None)
    assert out[2].tolist() == [0.0, INF, 0.0, 0.0, 0.0, 0.0, 0.0]
    keep = torch.tensor([0, 2, 3, 4, 5, 6], device=DEV)
    out = _policy(lp[keep], ol[keep], None, adv[keep], None)
    _one(out[0], -f32(0.28) - 1 + 2 * (1 - f32(0.2)), 4, "loss")


def test_policy_reference_beyond_reach():
    """KL terms of tokens that one policy cannot give are infinite, not NaN."""
    lp = torch.tensor([-INF, -1.0, -800.0], device=DEV)
    rf = torch.tensor([-1.0, -INF, 0.0], device=DEV)
    for i in range(3):
        out = _policy(lp[i:i + 1], None, rf[i:i + 1], torch.zeros(1, device=DEV), None, beta=1.0)
        assert out[0] == INF and out[1][1] == INF, i


@pytest.mark.parametrize("n", [5, 9000])
def test_policy_kl_only_watched(n):
    """With beta = 0 the KL terms are reported and enter neither the loss nor its
    gradient, infinities and NaN among them."""
    lp, ol, rf, adv, w = _policy_inputs(n, 21, weighted=False)
    want = _policy(lp, ol, None, adv, w, beta=0.0)
    for bad in (-INF, INF, NAN):
        rf[n // 2] = bad
        out = _policy(lp, ol, rf, adv, w, beta=0.0)
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]), bad
        assert torch.equal(out[1][::2], want[1][::2])
        assert torch.isnan(out[1][1]) if bad != bad else out[1][1] == INF, bad


def test_policy_no_tokens():
    e = torch.empty(0, device=DEV)
    out = _policy(e, e, e, e, e)
    assert not out[0].any() and not out[1].any()


# ---- preference loss -------------------------------------------------------------

def _pref(lp, off, rf=None, v=None, w=None, dloss=None, **kw):
    p = off.numel() // 2
    loss, rew = torch.full((1,), 7.0, device=DEV), torch.full((2 * p,), 7.0, device=DEV)
    g = torch.full_like(lp, 7.0)
    preference_loss(lp, off, loss, ref_logp=rf, valid=v, weight=w, rewards=rew, dlogp=g, dloss=dloss, **kw)
    return loss, rew, g


def _check_pref(lp, off, rf, v, w, out, beta=0.1, margin=0.0, smoothing=0.0, average=False, dloss=1.0):
    want, rew, g = R.preference_loss(h64(lp), _opt(rf), None if v is None else v.cpu().numpy(), off.cpu().numpy(), _opt(w),
                                     f32(beta), f32(margin), f32(smoothing), average, f32(dloss), np.full(lp.numel(), 7.0))
    size = np.abs(rew).sum() + abs(want) + 1
    _one(out[0], want, size, "loss")
    _one(out[1], rew, size, "rewards")
    _one(out[2], g, np.abs(g) * size + 1e-6, "dlogp")


def _answers(pairs, mean, seed, lead=0, tail=0):
    rng = np.random.Generator(np.random.PCG64(seed))
    lens = rng.integers(0, 2 * mean + 1, 2 * pairs)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]) + lead).to(DEV)
    n = int(lens.sum()) + lead + tail
    lp = -torch.exp(draw((n,), seed, 1.5, -1.5)).to(DEV)
    rf = (lp + draw((n,), seed + 1, 0.1).to(DEV)).clamp(max=0)
    return lp, rf, off


@pytest.mark.parametrize("pairs,mean", [(1, 1), (1, 40), (3, 7), (4, 300), (8, 250), (1, 2100), (8, 900), (9, 100), (40, 5), (3, 20000),
                                        (600, 30), (1, 200000)])
@pytest.mark.parametrize("average", [False, True])
def test_preference(pairs, mean, average):
    lp, rf, off = _answers(pairs, mean, pairs + mean, lead=3, tail=5)
    kw = dict(beta=1.5 if average else 0.1, margin=0.2, smoothing=0.1, average=average)
    out = _pref(lp, off, rf, **kw)
    _check_pref(lp, off, rf, None, None, out, **kw)
    assert (out[2][:3] == 7).all() and (out[2][-5:] == 7).all()  # no sequence holds them
    v = (draw((lp.numel(),), 77).to(DEV) > -0.5)
    w = torch.rand(pairs, generator=torch.Generator().manual_seed(3)).to(DEV)
    ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for valid in (v, v.to(torch.uint8)):
        out = _pref(lp, off, None, valid, w, dloss=torch.tensor([1.7], device=DEV), workspace=ws, **kw)
        _check_pref(lp, off, None, v, w, out, dloss=1.7, **kw)
    loss = torch.empty(1, device=DEV)
    preference_loss(lp, off, loss, valid=v, weight=w, **kw)
    assert torch.equal(loss, out[0])


def test_preference_padded_batch():
    """Answers as rows of a padded batch: offsets at the rows' ends, padding not valid."""
    p, t = 5, 64
    lp, rf = -torch.exp(draw((2 * p, t), 1)).to(DEV), -torch.exp(draw((2 * p, t), 2)).to(DEV)
    v = torch.arange(t, device=DEV)[None] < torch.tensor([64, 0, 1, 30, 63, 64, 5, 9, 64, 2], device=DEV)[:, None]
    off = torch.arange(0, (2 * p + 1) * t, t, device=DEV)
    want = _pref(lp, off, rf, v, average=True, beta=2.0)
    _check_pref(lp.flatten(), off, rf.flatten(), v.flatten(), None, [x.flatten() for x in want], average=True, beta=2.0)
    lp[~v], rf[~v] = NAN, INF
    got = _pref(lp, off, rf, v, average=True, beta=2.0)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[2][~v].any()


def test_preference_large_margins_and_smoothing():
    off = torch.tensor([0, 1, 2, 3, 4, 5, 6], device=DEV)
    lp = torch.tensor([-1.0, -900.0, -3e5, -900.0, -1.0, -3.0], device=DEV)
    for smoothing in (0.0, 0.3, 1.0):
        out = _pref(lp, off, beta=1.0, smoothing=smoothing)
        _check_pref(lp, off, None, None, None, out, beta=1.0, smoothing=smoothing)
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()


def test_preference_pairs_that_do_not_count():
    lp, rf, off = _answers(6, 50, 11)
    w = torch.tensor([0.5, 0.0, 0.3, 0.0, 0.2, 0.1], device=DEV)
    want = _pref(lp, off, rf, w=w)
    o = off.tolist()
    for s in (1, 3, 7, 9):
        lp[o[s]:o[s + 1]] = NAN
    got = _pref(lp, off, rf, w=w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    for s in (1, 3, 7, 9):
        assert not got[2][o[s]:o[s + 1]].any()


def test_preference_bad_offsets_stay_in_bounds():
    """Offsets before the first token, behind the last one or falling are no
    fault: a sequence is cut to the tokens that exist, or empty."""
    lp = -torch.rand(100, generator=torch.Generator().manual_seed(1)).to(DEV)
    for o in ([-5, 10, 400], [50, 20, 30], [0, 1 << 62, 1 << 62], [-(1 << 63), (1 << 63) - 1, 0], [200, 300, 400]):
        off = torch.tensor(o, device=DEV)
        out = _pref(lp, off)
        _check_pref(lp, off, None, None, None, out)


@pytest.mark.parametrize("pairs", [3, 40])
def test_preference_answers_beyond_reach(pairs):
    """An answer that the policy cannot give has the reward -inf: a pair whose
    rejected answer it is costs nothing without smoothing, one whose preferred
    answer it is costs nothing with a smoothing of 1."""
    n = 2 * pairs * 6
    off = torch.arange(0, n + 1, 6, device=DEV)
    lp = -torch.exp(draw((n,), 31)).to(DEV)
    w = torch.full((pairs,), 0.25, device=DEV)
    for seq, smoothing in ((pairs + 1, 0.0), (1, 1.0)):
        x, v = lp.clone(), w.clone()
        x[seq * 6 + 2], v[1] = -INF, 0.0
        want = _pref(lp, off, w=v, smoothing=smoothing)
        out = _pref(x, off, w=w, smoothing=smoothing)
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and out[1][seq] == -INF
        out = _pref(x, off, w=w, smoothing=1.0 - smoothing)
        assert out[0] == INF and not torch.isnan(out[2]).any()
        out = _pref(x, off, w=w, smoothing=0.125)
        assert out[0] == INF and not torch.isnan(out[2]).any()


def test_preference_nothing():
    lp = -torch.rand(10, generator=torch.Generator().manual_seed(1)).to(DEV)
    out = _pref(lp, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert out[0] == 0 and (out[2] == 7).all()
    e = torch.empty(0, device=DEV)
    out = _pref(e, torch.zeros(5, dtype=torch.int64, device=DEV), margin=0.5)
    _one(out[0], np.log1p(np.exp(0.5)), 1, "loss")
    assert not out[1].any()


def test_gradients_against_differences():
    n = 200
    lp, ol, rf, adv, w = _policy_inputs(n, 41)
    g = _policy(lp, ol, rf, adv, w)[2]
    v = h64(draw((n,), 42))
    f = lambda z: R.policy_loss(z, h64(ol), h64(rf), h64(adv), h64(w), f32(0.2), f32(0.28), f32(0.1))[0]
    num = (f(h64(lp) + 1e-6 * v) - f(h64(lp) - 1e-6 * v)) / 2e-6
    assert abs((h64(g) * v).sum() - num) < 1e-6
    lp, rf, off = _answers(4, 20, 43)
    g = _pref(lp, off, rf, beta=0.5, smoothing=0.1)[2]
    v = h64(draw((lp.numel(),), 44))
    f = lambda z: R.preference_loss(z, h64(rf), None, off.cpu().numpy(), None, f32(0.5), 0.0, f32(0.1), False)[0]
    num = (f(h64(lp) + 1e-6 * v) - f(h64(lp) - 1e-6 * v)) / 2e-6
    assert abs((h64(g) * v).sum() - num) < 1e-6


def test_refused_workspaces():
    a = _policy_inputs(6000, 51)
    with pytest.raises(MuonError) as e:
        _policy(*a, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    lp, rf, off = _answers(40, 5, 52)
    with pytest.raises(MuonError) as e:
        _pref(lp, off, rf, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5


def test_graph_replays_and_streams():
    n = 30000
    sets = [_policy_inputs(n, 61 + 10 * i) for i in range(3)]
    lp0, rf, off = _answers(20, n // 40, 62)
    cur = [t.clone() for t in sets[0]]
    m = lp0.numel()
    prefs = [(-torch.exp(draw((m,), 95 + i))).to(DEV) for i in range(3)]
    plp = prefs[0].clone()
    new = lambda: [torch.zeros(1, device=DEV), torch.zeros(3, device=DEV), torch.zeros(n, device=DEV),
                   torch.zeros(1, device=DEV), torch.zeros(40, device=DEV), torch.zeros(m, device=DEV)]

    def step(a, p, o, stream=None):
        policy_loss(a[0], a[1], a[3], o[0], ref_logp=a[2], weight=a[4], dlogp=o[2], terms=o[1], beta=0.1, stream=stream)
        preference_loss(p, off, o[3], ref_logp=rf, rewards=o[4], dlogp=o[5], stream=stream)

    rec = new()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(cur, plp, rec)
    side = torch.cuda.Stream()
    for i in (0, 1, 2, 1, 0):
        for c, s in zip(cur, sets[i]):
            c.copy_(s)
        plp.copy_(prefs[i])
        graph.replay()
        torch.cuda.synchronize()
        o = new()
        torch.cuda.synchronize()
        step(sets[i], prefs[i], o, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, rec))
