"""GPU token log-probabilities and their gradient against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import MuonError, token_logp, token_logp_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def _run(x, t, scale=1.0, **kw):
    logp, lse = (torch.full((x.shape[0],), 7.0, device=DEV) for _ in range(2))
    token_logp(x, t, logp, lse, scale=scale, **kw)
    return logp, lse


def _check(x, t, scale, logp, lse):
    """Bounds: a term exp(z - m) is off by three roundings of z - m and two of
    itself; the sum over the others by that on average (weighted by the terms)
    and by its chain of additions, at most vocab / 64 in a thread, each with a
    rescaling, and 20 joins."""
    xs, ts = h64(x), t.cpu().numpy()
    sc = float(np.float32(scale))
    wl, ws = R.token_logp(xs, ts, sc)
    chain = 1.25 * xs.shape[1] / (64 if xs.shape[1] <= 2048 else 256) + 40
    bl, bs = np.zeros_like(wl), np.zeros_like(ws)
    for i, at in enumerate(ts):
        if not 0 <= at < xs.shape[1] or not np.isfinite(ws[i]):
            continue
        z = xs[i] * sc
        m = z.max()
        d = m - z
        e = np.exp(-d)
        with np.errstate(invalid="ignore"):
            de = np.where(e > 0, e * np.where(np.isfinite(d), d, 0.0), 0.0)
        rest = np.delete(e, at).sum()
        rel = (3 * np.delete(de, at).sum() / max(rest, 1e-300) + chain) * U
        own = (3 * d[at] + 6) * U
        if rest < e[at]:
            bl[i] = (rel + own + 6 * U) * abs(wl[i]) + 1e-37
        elif np.isfinite(d[at]):
            bl[i] = rel + own + 6 * U * abs(wl[i])
        mine = own * min(1.0, e[at]) if e[at] > 0 else 0.0  # (d + 2) e^-d goes to 0
        bs[i] = rel + mine + 4 * U + 2 * U * abs(ws[i]) + 2 * U * abs(m)
    ok = np.isfinite(wl)
    within(logp[torch.from_numpy(ok).to(DEV)], wl[ok], bl[ok], "logp")
    assert np.array_equal(h64(logp)[~ok], wl[~ok])
    ok = np.isfinite(ws)
    within(lse[torch.from_numpy(ok).to(DEV)], ws[ok], bs[ok], "lse")
    assert np.array_equal(h64(lse)[~ok], ws[~ok])
    return wl, ws


def _check_grad(x, t, scale, logp, lse, dlogp, out):
    xs, ts = h64(x), t.cpu().numpy()
    sc = float(np.float32(scale))
    with np.errstate(invalid="ignore", over="ignore"):
        want = R.token_logp_backward(xs, ts, sc, h64(logp), h64(lse), h64(dlogp))
        away = np.abs(xs * sc - h64(lse)[:, None])
    # three roundings of z - lse, and a few of the product
    rel = 3 * np.where(np.isfinite(away), away, 0.0) + 12
    within(out, want, half_step(out.dtype) * np.abs(want) * (1 + 1e-6) + rel * U * np.abs(want) * 1.01, "dlogits")


def _logits(rows, vocab, dt, seed, std=3.0):
    return draw((rows, vocab), seed, std, 0.0, DTYPES[dt]).to(DEV)


def _targets(rows, vocab, seed, ignored=0.2):
    rng = np.random.Generator(np.random.PCG64(seed))
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < ignored] = -100
    return torch.from_numpy(t).to(DEV)


VOCABS = [1, 2, 3, 7, 8, 9, 63, 64, 65, 100, 511, 512, 513, 1000, 2047, 2048, 2049, 4096, 5003, 8191, 8192, 8200, 16384,
          16385, 20000, 33001, 50021, 65536, 65537, 80000]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_vocabularies(vocab, dt):
    for rows, scale in ((1, 1.0), (6, 0.7), (530 if vocab <= 1000 else 33, 1.25)):
        x, t = _logits(rows, vocab, dt, vocab + rows), _targets(rows, vocab, vocab + rows, 0.2 if rows > 1 else 0.0)
        logp, lse = _run(x, t, scale)
        _check(x, t, scale, logp, lse)
        d = draw((rows,), 3, 0.5).to(DEV)
        dx = torch.full_like(x, 5.0)
        token_logp_backward(x, t, logp, lse, d, dx, scale=scale)
        _check_grad(x, t, scale, logp, lse, d, dx)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [100, 5000, 40000])
def test_nearly_certain_targets(vocab, dt):
    """Log-probabilities down to far below the last place of 1 keep their
    relative accuracy, and so does the target's own gradient."""
    rows = 24
    x, t = _logits(rows, vocab, dt, 5, 1.0), _targets(rows, vocab, 6, 0.0)
    for i in range(rows):
        x[i, t[i]] = 2.0 * i
    logp, lse = _run(x, t)
    want, _ = _check(x, t, 1.0, logp, lse)
    assert want.max() > -1e-14 and (h64(logp) < 0).all()
    d, dx = torch.ones(rows, device=DEV), torch.empty_like(x)
    token_logp_backward(x, t, logp, lse, d, dx)
    _check_grad(x, t, 1.0, logp, lse, d, dx)
    own = h64(dx.gather(1, t[:, None]))[:, 0]
    exact = -np.expm1(want)
    assert (np.abs(own - exact) <= (half_step(x.dtype) * 1.01 + 400 * U) * exact + 1e-37).all()


def test_unlikely_targets():
    x, t = _logits(20, 3000, "f32", 7), _targets(20, 3000, 8, 0.0)
    for i in range(20):
        x[i, t[i]] = -float(10 ** (i / 3))
    x[3, t[3]] = -INF
    x[4, t[4]] = -3.4e38
    logp, lse = _run(x, t)
    _check(x, t, 1.0, logp, lse)
    assert logp[3] == -INF and logp[4] < -3e38


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,rows", [(70, 40), (3000, 40), (30000, 20), (30000, 600), (70000, 20)])
def test_masks(vocab, rows, dt):
    """Words that cannot be, rows without any, rows at the type's lowest value,
    and rows whose values nobody counts."""
    lowest = torch.finfo(DTYPES[dt]).min
    x, t = _logits(rows, vocab, dt, 9), _targets(rows, vocab, 10, 0.3)
    shut = torch.rand(rows, vocab, generator=torch.Generator().manual_seed(1)).to(DEV) < 0.5
    shut[torch.arange(rows), t.clamp(min=0)] = False
    x[shut] = -INF
    x[2], x[3], x[4] = -INF, -INF, lowest
    t[2], t[3], t[4] = 1, vocab - 1, 5
    x[3, vocab - 1] = 0.5      # the target alone is left
    x[5] = -INF
    x[5, 7], t[5] = 1.0, 8     # another word alone is left
    x[6, : vocab // 2] = lowest
    t[7], t[8], t[9] = vocab, -1, 1 << 40
    none = (t < 0) | (t >= vocab)
    clean = x.clone()
    x[none] = NAN
    logp, lse = _run(x, t)
    _check(clean, t, 1.0, logp, lse)
    assert logp[2] == 0 and lse[2] == -INF and logp[3] == 0 and lse[3] == 0.5 and logp[5] == -INF and lse[5] == 1.0
    # some term of a row at the lowest value is 1 each: the probability is 1 / vocab
    assert abs(float(logp[4]) + np.log(vocab)) < 1e-5
    assert not logp[none].any() and not lse[none].any()
    d = draw((rows,), 11).to(DEV)
    d[12:16] = 0.0
    x[13] = NAN                # not read
    dx = torch.full_like(x, 5.0)
    token_logp_backward(x, t, logp, lse, d, dx)
    assert not dx[none].any() and not dx[2].any() and not dx[12:16].any()
    rows_left = torch.ones(rows, dtype=torch.bool, device=DEV)
    rows_left[[4, 5]] = False  # lse of row 4 cannot hold log(vocab); the target of row 5 cannot be
    _check_grad(clean[rows_left], t[rows_left], 1.0, logp[rows_left], lse[rows_left], d[rows_left], dx[rows_left])
    assert not dx[shut & rows_left[:, None] & ~none[:, None]].any()


def test_bad_values_stay_in_their_rows():
    for vocab in (90, 4000, 30000, 70000):
        x, t = _logits(30, vocab, "f32", 12), _targets(30, vocab, 13, 0.0)
        want = _run(x, t)
        y = x.clone()
        y[3, 4], y[5, vocab - 1], y[7] = NAN, INF, NAN
        y[9, t[9]] = NAN
        y[11, t[11]] = INF
        y[13] = -INF
        y[13, t[13]] = NAN
        got = _run(y, t)
        bad = torch.zeros(30, dtype=torch.bool, device=DEV)
        bad[[3, 5, 7, 9, 11, 13]] = True
        for a, b in zip(got, want):
            assert torch.isnan(a[bad]).all() and torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 33000), (3, 70001), (2, 140000), (100, 20011), (700, 3001), (3000, 130)])
def test_strides_workspaces_and_repeats(rows, vocab, dt):
    x, t = _logits(rows, vocab, dt, 14), _targets(rows, vocab, 15)
    want = _run(x, t, 0.9)
    if rows <= 100:
        _check(x, t, 0.9, *want)
    buf = torch.full((rows * (vocab + 3) + 1,), 3.0, dtype=DTYPES[dt], device=DEV)
    v = buf[1:].view(rows, vocab + 3)[:, :vocab]
    v.copy_(x)
    ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(workspace=ws), dict(workspace=ws)):
        assert all(torch.equal(a, b) for a, b in zip(_run(v, t, 0.9, **kw), want))
    d = draw((rows,), 16).to(DEV)
    dx = torch.empty_like(x)
    token_logp_backward(x, t, *want, d, dx, scale=0.9)
    # in place, among other values
    token_logp_backward(v, t, *want, d, v, scale=0.9)
    assert torch.equal(v, dx)
    v.fill_(3.0)
    assert (buf == 3.0).all()
    if rows <= 3 and vocab > 65536:  # rows that several workgroups share
        with pytest.raises(MuonError) as e:
            _run(x, t, workspace=ws[:16])
        assert e.value.status == 5


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [4097, 16387])
@pytest.mark.parametrize("vocab", [1, 5, 64, 65, 100, 128, 129, 256, 257, 500, 512, 700, 1000, 1024])
def test_many_short_rows(vocab, rows, dt):
    """Rows that a wave takes several of, whole: values, masks and strides as in
    the other forms."""
    x, t = _logits(rows, vocab, dt, 71), _targets(rows, vocab, 72, 0.3)
    if vocab > 4:
        x[torch.rand(rows, vocab, generator=torch.Generator().manual_seed(2)).to(DEV) < 0.2] = -INF
        x[torch.arange(rows, device=DEV), t.clamp(min=0)] = 1.0
        x[1], x[2], x[5] = -INF, -INF, 0.0
        t[1], t[2] = 0, vocab - 1
        x[2, vocab - 1] = 0.5
    none = t < 0
    clean = x.clone()
    x[none] = NAN
    buf = torch.full((rows * (vocab + 3) + 1,), 3.0, dtype=DTYPES[dt], device=DEV)
    v = buf[1:].view(rows, vocab + 3)[:, :vocab]
    v.copy_(x)
    logp, lse = _run(x, t, 0.9)
    assert all(torch.equal(a, b) for a, b in zip(_run(v, t, 0.9), (logp, lse)))
    assert not logp[none].any() and not lse[none].any()
    part = torch.arange(0, rows, 37, device=DEV)
    part = torch.cat([part, torch.tensor([1, 2, 5, rows - 1], device=DEV)])
    _check(clean[part], t[part], 0.9, logp[part], lse[part])
    bad = x.clone()
    bad[8, vocab // 2], t[8] = NAN, 0
    got = _run(bad, t, 0.9)
    assert torch.isnan(got[0][8]) and torch.equal(got[0][9:12], logp[9:12]) and torch.equal(got[1][:8], lse[:8])


def test_activations_of_three_dimensions():
    x = _logits(12, 50, "f32", 17).view(3, 4, 50)
    t = _targets(12, 50, 18).view(3, 4)
    logp, lse = torch.empty(3, 4, device=DEV), torch.empty(3, 4, device=DEV)
    token_logp(x, t, logp, lse)
    a, b = _run(x.view(12, 50), t.view(12))
    assert torch.equal(logp.view(12), a) and torch.equal(lse.view(12), b)


def test_rows_beyond_32_bit_offsets():
    ld, vocab = (1 << 31) + 8, 20000
    buf = torch.empty(2 * ld + vocab, dtype=torch.bfloat16, device=DEV)
    v = buf.as_strided((3, vocab), (ld, 1))
    x, t = _logits(3, vocab, "bf16", 19), _targets(3, vocab, 20, 0.0)
    v.copy_(x)
    want = _run(x, t)
    assert all(torch.equal(a, b) for a, b in zip(_run(v, t), want))
    dx, d = torch.empty_like(x), torch.ones(3, device=DEV)
    token_logp_backward(x, t, *want, d, dx)
    token_logp_backward(v, t, *want, d, v)
    assert torch.equal(v, dx)


def test_many_rows_of_few_words():
    """More rows than one launch has workgroups for."""
    rows, vocab = 300001, 9
    x, t = _logits(rows, vocab, "bf16", 91), _targets(rows, vocab, 92)
    logp, lse = _run(x, t)
    d = draw((rows,), 93).to(DEV)
    dx = torch.full_like(x, 5.0)
    token_logp_backward(x, t, logp, lse, d, dx)
    part = torch.cat([torch.arange(0, rows, 3001, device=DEV), torch.tensor([rows - 1, 262143, 262144], device=DEV)])
    _check(x[part], t[part], 1.0, logp[part], lse[part])
    _check_grad(x[part], t[part], 1.0, logp[part], lse[part], d[part], dx[part])
    again = torch.empty_like(x[200000:])
    token_logp_backward(x[200000:], t[200000:], logp[200000:], lse[200000:], d[200000:], again)
    assert torch.equal(again, dx[200000:])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_logits(dt):
    """Logits and gradients beyond what the caches hold: the same bits as part by
    part."""
    vocab = 30011
    rows = (260 << 20) // (vocab * (4 if dt == "f32" else 2))
    x = torch.empty(rows, vocab, dtype=DTYPES[dt], device=DEV)
    x.copy_(_logits(64, vocab, dt, 94).repeat(rows // 64 + 1, 1)[:rows])
    t, d = _targets(rows, vocab, 95), draw((rows,), 96).to(DEV)
    logp, lse = _run(x, t)
    dx = torch.empty_like(x)
    token_logp_backward(x, t, logp, lse, d, dx)
    _check(x[:40], t[:40], 1.0, logp[:40], lse[:40])
    for at in (0, rows - 600):
        s = slice(at, at + 600)
        a, b = _run(x[s], t[s])
        assert torch.equal(a, logp[s]) and torch.equal(b, lse[s])
        again = torch.empty_like(x[s])
        token_logp_backward(x[s], t[s], a, b, d[s], again)
        assert torch.equal(again, dx[s])
    token_logp_backward(x, t, logp, lse, d, x)
    assert torch.equal(x, dx)


def test_gradient_against_differences():
    rows, vocab, scale = 7, 31, 1.5
    x, t = _logits(rows, vocab, "f32", 21), _targets(rows, vocab, 22, 0.3)
    logp, lse = _run(x, t, scale)
    d = draw((rows,), 23).to(DEV)
    dx = torch.empty_like(x)
    token_logp_backward(x, t, logp, lse, d, dx, scale=scale)
    v = h64(draw((rows, vocab), 24))
    f = lambda z: (R.token_logp(z, t.cpu().numpy(), scale)[0] * h64(d)).sum()
    num = (f(h64(x) + 1e-5 * v) - f(h64(x) - 1e-5 * v)) / 2e-5
    assert abs((h64(dx) * v).sum() - num) <= 1e-7 + 100 * U * np.abs(v).sum() * np.abs(h64(d)).max() * scale
    # probabilities add to one: a row's gradients add to nothing
    assert np.abs(h64(dx).sum(1)).max() <= 100 * U * np.abs(h64(d)).max() * scale * 2


def test_no_tokens():
    x, t, f = torch.empty(0, 9, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    token_logp(x, t, f, f.clone())
    token_logp_backward(x, t, f, f.clone(), f.clone(), x.clone())


def test_graph_replays_and_streams():
    for rows, vocab in ((5, 80000), (5, 40000), (700, 3000)):
        xs = [_logits(rows, vocab, "bf16", 31 + i) for i in range(3)]
        t, d = _targets(rows, vocab, 35), draw((rows,), 36).to(DEV)
        x = xs[0].clone()
        new = lambda: [torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV), torch.zeros_like(x)]

        def step(src, o, stream=None):
            token_logp(src, t, o[0], o[1], stream=stream)
            token_logp_backward(src, t, o[0], o[1], d, o[2], stream=stream)

        rec = new()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step(x, rec)
        side = torch.cuda.Stream()
        for src in xs + xs:
            x.copy_(src)
            graph.replay()
            torch.cuda.synchronize()
            o = new()
            torch.cuda.synchronize()
            step(src, o, stream=side)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, rec))
