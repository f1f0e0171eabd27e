"""GPU norm and rotation of query and key heads, forward and backward, against
the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import MuonError, qk_norm_rope, qk_norm_rope_backward
from oracle import ends_ref as R
from tests.ops_helpers import DEV, DTYPES, K, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _layout(kind, b, t, h, d, dt, others=3):
    """(empty tensor [b, t, h, d] in a layout, the buffer around it)."""
    if kind == "packed":      # a slice of a projection's output
        buf = torch.full((b, t, h + others, d), 3.0, dtype=dt, device=DEV)
        return buf[:, :, 1:1 + h], buf
    if kind == "heads":       # heads before tokens
        buf = torch.full((b, h, t, d), 3.0, dtype=dt, device=DEV)
        return buf.transpose(1, 2), buf
    if kind == "tokens":      # tokens before sequences
        buf = torch.full((t, b, h, d), 3.0, dtype=dt, device=DEV)
        return buf.transpose(0, 1), buf
    if kind == "mixed":       # query, key and value of a head side by side, at an odd address
        buf = torch.full((1 + b * t * h * 3 * d,), 3.0, dtype=dt, device=DEV)
        return buf[1:].view(b, t, h, 3, d)[:, :, :, 1], buf
    return (torch.full((b, t, h, d), 3.0, dtype=dt, device=DEV),) * 2


def _in(kind, values, dt):
    t, buf = _layout(kind, *values.shape, DTYPES[dt])
    t.copy_(values.to(DTYPES[dt]))
    return t


def _angles(rot, rows=97):
    c, s = R.table(rows, rot)
    if rot == 0:
        return None, None, c, s
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), c, s


def _check_fwd(out, x, gamma, c, s, rot, inter, what):
    xs, g = h64(x), None if gamma is None else h64(gamma)
    want = R.qk_norm_rope(xs, g, c, s, rot, inter, EPS)
    # roundings of the two products that an element is the sum of
    mag = np.abs(R.qk_norm_rope(xs, g, np.ones_like(c), np.zeros_like(s), rot, inter, EPS))
    mag = R.turn(mag, np.abs(c), -np.abs(s), rot, inter)
    i, j = R.pairs(rot, inter)
    y = np.abs(R.qk_norm_rope(xs, g, np.ones_like(c), np.zeros_like(s), rot, inter, EPS))
    mag[..., j] = y[..., j] * np.abs(c) + y[..., i] * np.abs(s)
    within(out, want, half_step(out.dtype) * np.abs(want) * (1 + 1e-6) + K * U * mag, what)


def _check_bwd(dx, dgamma, dy, x, gamma, c, s, rot, inter, what):
    xs, g, ds = h64(x), None if gamma is None else h64(gamma), h64(dy)
    want, wgamma = R.qk_norm_rope_backward(ds, xs, g, c, s, rot, inter, EPS)
    r = 1 / np.sqrt((xs ** 2).mean(-1, keepdims=True) + EPS)
    xh = np.abs(xs) * r
    back = np.abs(ds)
    i, j = R.pairs(rot, inter)
    mag = back.copy()
    mag[..., i] = back[..., i] * np.abs(c) + back[..., j] * np.abs(s)
    mag[..., j] = back[..., j] * np.abs(c) + back[..., i] * np.abs(s)
    gm = mag if g is None else mag * np.abs(g)
    inner = r * (gm + xh * (gm * xh).mean(-1, keepdims=True))
    within(dx, want, half_step(dx.dtype) * np.abs(want) * (1 + 1e-6) + K * U * inner, what)
    if dgamma is not None:
        # a lane's rows, 10 joins in the workgroup, and at most 1024 / 32 + 32 of the workgroups' sums
        chain = x[..., 0].numel() / 4096 + 16 + 10 + 64 + K
        within(dgamma, wgamma, half_step(dgamma.dtype) * np.abs(wgamma) * (1 + 1e-6)
               + chain * U * (mag * xh).reshape(-1, xs.shape[-1]).sum(0), what + " gain")


def _case(dim, rot, inter, dt, wdt, b=2, t=5, hq=3, hk=1, lx="plain", ly="plain", positions=None, gains=True, seed=1):
    q, k = (_in(lx, draw((b, t, h, dim), seed + i, 1.3, 0.2), dt) for i, h in enumerate((hq, hk)))
    dqo, dko = (_in(ly, draw((b, t, h, dim), seed + 5 + i, 0.4), dt) for i, h in enumerate((hq, hk)))
    gq, gk = (draw((dim,), seed + 10 + i, 0.3, 1.0, DTYPES[wdt]).to(DEV) if gains else None for i in range(2))
    cos, sin, cn, sn = _angles(rot, max(97, t) if positions is None else 97)
    pos = None if positions is None else torch.as_tensor(positions).to(DEV)
    c, s = R.token_angles(cn, sn, rot, b, t, None if pos is None else pos.cpu().numpy())
    kw = dict(positions=pos, interleaved=inter, eps=EPS)
    (qo, qb), (ko, kb) = (_layout(ly, b, t, h, dim, DTYPES[dt]) for h in (hq, hk))
    qk_norm_rope(q, k, gq, gk, cos, sin, qo, ko, **kw)
    _check_fwd(qo, q, gq, c, s, rot, inter, "q_out")
    _check_fwd(ko, k, gk, c, s, rot, inter, "k_out")
    (dq, dqb), (dk, dkb) = (_layout(lx, b, t, h, dim, DTYPES[dt]) for h in (hq, hk))
    dgq, dgk = (torch.full((dim,), 5.0, dtype=DTYPES[wdt], device=DEV) for _ in range(2))
    qk_norm_rope_backward(dqo, dko, q, k, gq, gk, cos, sin, dq, dk, dgamma_q=dgq, dgamma_k=dgk, **kw)
    _check_bwd(dq, dgq, dqo, q, gq, c, s, rot, inter, "dq")
    _check_bwd(dk, dgk, dko, k, gk, c, s, rot, inter, "dk")
    res = [v.clone() for v in (qo, ko, dq, dk, dgq, dgk)]
    for view, buf in ((qo, qb), (ko, kb), (dq, dqb), (dk, dkb)):
        view.fill_(3.0)
        assert (buf == 3.0).all(), "elements between the heads were written"
    return res


DIMS = [(1, 0), (2, 2), (3, 2), (7, 4), (8, 8), (15, 14), (16, 16), (16, 8), (20, 20), (31, 10), (32, 32), (48, 16),
        (64, 64), (64, 32), (66, 66), (80, 40), (80, 80), (96, 96), (112, 112), (127, 0), (128, 128), (128, 64), (128, 2),
        (160, 96), (192, 64), (200, 200), (255, 254), (256, 256), (256, 18), (320, 320), (384, 128), (511, 130), (512, 512),
        (512, 2)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", DIMS)
def test_dims(dim, rot, inter, dt):
    _case(dim, rot, inter, dt, "f32" if dim % 3 else "bf16")
    _case(dim, rot, inter, dt, dt, b=1, t=37, hq=4, hk=3, lx="packed", ly="heads")


@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("lx", ["plain", "packed", "heads", "tokens", "mixed"])
def test_layouts_give_the_same_bits(lx, dt, wdt):
    for dim, rot, inter in ((64, 64, False), (80, 40, True), (36, 22, False)):
        a = _case(dim, rot, inter, dt, wdt, b=3, t=11, hq=6, hk=2)
        for ly in ("plain", "heads", "mixed"):
            b = _case(dim, rot, inter, dt, wdt, b=3, t=11, hq=6, hk=2, lx=lx, ly=ly)
            # the gains' sums take the rows in the order of memory
            assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))


@pytest.mark.parametrize("b,t,hq,hk", [(1, 1, 1, 1), (1, 1, 32, 8), (7, 1, 5, 1), (1, 613, 3, 3), (2, 1, 1, 130)])
def test_few_and_many_heads(b, t, hq, hk):
    _case(128, 128, False, "bf16", "bf16", b=b, t=t, hq=hq, hk=hk, positions=np.arange(t) % 97)
    _case(64, 24, True, "f32", "f32", b=b, t=t, hq=hq, hk=hk)


def test_many_rows():
    _case(64, 64, False, "bf16", "f32", b=2, t=6007, hq=8, hk=3, lx="packed", positions=np.arange(12014).reshape(2, 6007) % 90)
    _case(16, 16, True, "f32", "f32", b=1, t=40001, hq=5, hk=1, positions=np.arange(40001) % 97)


def test_positions():
    """Positions of each sequence or common to all; a token whose row does not
    exist is not turned."""
    far = np.array([[0, 96, 97, -1, 5], [1 << 40, -(1 << 62), 3, (1 << 63) - 1, 2]])
    for inter in (False, True):
        for rot in (32, 20):
            _case(32, rot, inter, "f32", "f32", positions=far)
            _case(32, rot, inter, "bf16", "f32", positions=far[0])
    wide = torch.arange(40, device=DEV).reshape(2, 20)
    q = draw((2, 5, 3, 32), 3).to(DEV)
    cos, sin, cn, sn = _angles(32)
    out, want = torch.empty_like(q), torch.empty_like(q)
    qk_norm_rope(q, None, None, None, cos, sin, out, None, positions=wide[:, 4:9], eps=EPS)
    qk_norm_rope(q, None, None, None, cos, sin, want, None, positions=wide[:, 4:9].contiguous(), eps=EPS)
    assert torch.equal(out, want)
    # a table without rows turns nothing, one that ends early those that have a row
    at = torch.arange(5, device=DEV)
    qk_norm_rope(q, None, None, None, cos[:0], sin[:0], out, None, positions=at, eps=EPS)
    # (not the bits of a call without a table, whose lanes hold other elements: the squares' sum has another order)
    qk_norm_rope(q, None, None, None, cos, sin, want, None, positions=torch.full((5,), -1, device=DEV), eps=EPS)
    assert torch.equal(out, want)
    qk_norm_rope(q, None, None, None, cos[:3].contiguous(), sin[:3].contiguous(), out, None, positions=at, eps=EPS)
    assert torch.equal(out[:, 3:], want[:, 3:]) and not torch.equal(out[:, 1:3], want[:, 1:3])
    with pytest.raises(MuonError) as e:  # without positions every token has to have a row
        qk_norm_rope(q, None, None, None, cos[:3].contiguous(), sin[:3].contiguous(), out, None, eps=EPS)
    assert e.value.status == 2


def test_far_positions():
    """Angles of far positions are the table's, whatever their size."""
    n = 1 << 20
    ang = (np.arange(n - 4, n)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64))
    cn, sn = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    cos, sin = torch.zeros(n, 32, device=DEV), torch.zeros(n, 32, device=DEV)
    cos[-4:], sin[-4:] = torch.from_numpy(cn).to(DEV), torch.from_numpy(sn).to(DEV)
    q = draw((1, 4, 2, 64), 5).to(DEV)
    out = torch.empty_like(q)
    qk_norm_rope(q, None, None, None, cos, sin, out, None, positions=torch.arange(n - 4, n, device=DEV), eps=EPS)
    _check_fwd(out, q, None, cn[None, :, None].astype(float), sn[None, :, None].astype(float), 64, False, "far")


def test_three_dimensions_and_queries_alone():
    q, k = draw((9, 4, 48), 1).to(DEV), draw((9, 2, 48), 2).to(DEV)
    g = draw((48,), 3, 0.1, 1.0).to(DEV)
    cos, sin, _, _ = _angles(48)
    a, b = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(q, k, g, None, cos, sin, a, b, eps=EPS)
    a4, b4 = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(q[None], k[None], g, None, cos, sin, a4[None], b4[None], eps=EPS)
    assert torch.equal(a, a4) and torch.equal(b, b4)
    alone = torch.empty_like(q)
    qk_norm_rope(q, None, g, None, cos, sin, alone, None, eps=EPS)
    assert torch.equal(a, alone)
    da, dk, db, d1 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty(48, device=DEV)
    d2 = torch.empty(48, device=DEV)
    qk_norm_rope_backward(a, b, q, k, g, None, cos, sin, da, dk, dgamma_q=d1, eps=EPS)
    qk_norm_rope_backward(a, None, q, None, g, None, cos, sin, db, None, dgamma_q=d2, eps=EPS)
    assert torch.equal(da, db)
    # nobody asks for the gains' gradients: the others are the same
    qk_norm_rope_backward(a, b, q, k, g, None, cos, sin, db, dk, eps=EPS)
    assert torch.equal(da, db)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (80, 40), (36, 22), (128, 128)])
def test_in_place(dim, rot, inter):
    cos, sin, _, _ = _angles(rot)
    buf = draw((2, 50, 9, dim), 7).to(DEV).bfloat16()
    q, k = buf[:, :, :6], buf[:, :, 6:8]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(q, k, None, None, cos, sin, qo, ko, interleaved=inter)
    d = draw((2, 50, 8, dim), 8).to(DEV).bfloat16()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope_backward(d[:, :, :6], d[:, :, 6:], q, k, None, None, cos, sin, dq, dk, interleaved=inter)
    qk_norm_rope_backward(d[:, :, :6], d[:, :, 6:], q, k, None, None, cos, sin, d[:, :, :6], d[:, :, 6:], interleaved=inter)
    assert torch.equal(d, torch.cat([dq, dk], 2))
    last = buf[:, :, 8].clone()
    qk_norm_rope(q, k, None, None, cos, sin, q, k, interleaved=inter)
    assert torch.equal(buf, torch.cat([qo, ko, last[:, :, None]], 2))


def test_extreme_rows():
    """Zero, constant, tiny and large heads; NaN and infinity stay in their own
    head."""
    x = draw((1, 8, 1, 64), 9).to(DEV)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 0.0, 7.0, 1e-20, x[0, 3] * 1e15
    cos, sin, cn, sn = _angles(64)
    c, s = R.token_angles(cn, sn, 64, 1, 8)
    out, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device=DEV)
    g = draw((64,), 10, 0.2, 1.0).to(DEV)
    dy = draw((1, 8, 1, 64), 11).to(DEV)
    for inter in (False, True):
        qk_norm_rope(x, None, g, None, cos, sin, out, None, interleaved=inter, eps=EPS)
        _check_fwd(out, x, g, c, s, 64, inter, "out")
        qk_norm_rope_backward(dy, None, x, None, g, None, cos, sin, dx, None, dgamma_q=dg, interleaved=inter, eps=EPS)
        _check_bwd(dx, dg, dy, x, g, c, s, 64, inter, "dx")
        y = x.clone()
        y[0, 5, 0, 3], y[0, 6, 0, 60] = float("nan"), float("inf")
        o2, d2 = torch.empty_like(x), torch.empty_like(x)
        qk_norm_rope(y, None, g, None, cos, sin, o2, None, interleaved=inter, eps=EPS)
        qk_norm_rope_backward(dy, None, y, None, g, None, cos, sin, d2, None, interleaved=inter, eps=EPS)
        keep = [0, 1, 2, 3, 4, 7]
        assert torch.equal(o2[0, keep], out[0, keep]) and torch.equal(d2[0, keep], dx[0, keep])
        assert torch.isnan(o2[0, 5]).all() and torch.isnan(o2[0, 6, 0, 60])
    # a small eps: 1 / sqrt(eps) ** 3 is beyond fp32, the gradient of a zero head is not
    for eps in (1e-30, 1e-44):
        zero = torch.zeros_like(x)
        qk_norm_rope(zero, None, g, None, cos, sin, out, None, eps=eps)
        assert not out.any()
        qk_norm_rope_backward(dy, None, zero, None, g, None, None, None, dx, None, eps=eps)
        e = float(np.float32(eps))
        want, _ = R.qk_norm_rope_backward(h64(dy), np.zeros(x.shape), h64(g), *R.token_angles(cn, sn, 0, 1, 8), 0, False, e)
        within(dx, want, 8 * U * np.abs(want), "tiny eps")


def test_slices_of_tokens_of_a_packed_buffer():
    """Some tokens of a projection's output, in place and into another buffer's:
    queries and keys lie between one another and do not overlap."""
    cos, sin, _, _ = _angles(32)
    buf = draw((3, 20, 7, 32), 51).to(DEV)
    part = buf[:, 4:15]
    q, k = part[:, :, :4], part[:, :, 4:6]
    qo, ko = torch.empty(3, 11, 4, 32, device=DEV), torch.empty(3, 11, 2, 32, device=DEV)
    qk_norm_rope(q, k, None, None, cos, sin, qo, ko)
    other = torch.full_like(buf, 3.0)
    to = other[:, 9:]
    qk_norm_rope(q, k, None, None, cos, sin, to[:, :, 2:6], to[:, :, :2])
    assert torch.equal(to[:, :, 2:6], qo) and torch.equal(to[:, :, :2], ko)
    to[:, :, :6] = 3.0
    assert (other == 3.0).all()
    with pytest.raises(MuonError):
        qk_norm_rope(q, k, None, None, cos, sin, to[:, :, 2:6], to[:, :, 5:7])
    want = buf.clone()
    want[:, 4:15, :4], want[:, 4:15, 4:6] = qo, ko
    qk_norm_rope(q, k, None, None, cos, sin, q, k)
    assert torch.equal(buf, want)


def test_heads_beyond_32_bit_offsets():
    big = (1 << 31) + 64
    store = torch.empty(big * 2 + 4096, dtype=torch.bfloat16, device=DEV)
    x = draw((3, 2, 4, 64), 61).to(DEV).bfloat16()
    cos, sin, _, _ = _angles(64)
    want, back, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device=DEV)
    g = draw((64,), 62, 0.1, 1.0).to(DEV)
    qk_norm_rope(x, None, g, None, cos, sin, want, None)
    qk_norm_rope_backward(want, None, x, None, g, None, cos, sin, back, None, dgamma_q=dg)
    v = store.as_strided((3, 2, 4, 64), (big, 4 * 64, 64, 1))
    v.copy_(x)
    got, d2, dg2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(dg)
    qk_norm_rope(v, None, g, None, cos, sin, got, None)
    assert torch.equal(got, want)
    qk_norm_rope_backward(want, None, v, None, g, None, cos, sin, d2, None, dgamma_q=dg2)
    assert torch.equal(d2, back) and torch.equal(dg2, dg)
    qk_norm_rope(v, None, g, None, cos, sin, v, None)
    assert torch.equal(v, want)


def test_large_outputs():
    """Outputs beyond what the caches hold take other stores: the same bits."""
    for dt in ("bf16", "f32"):
        x = draw((1, 1, 8, 128), 71, 1.0, 0.0, DTYPES[dt]).to(DEV)
        cos, sin, _, _ = _angles(128)
        n = (100 << 20) // (8 * 128 * x.element_size())
        many = x.expand(1, n, 8, 128).contiguous()
        pos = torch.full((n,), 7, device=DEV)
        one, out = torch.empty_like(x), torch.empty_like(many)
        qk_norm_rope(x, None, None, None, cos, sin, one, None, positions=pos[:1])
        qk_norm_rope(many, None, None, None, cos, sin, out, None, positions=pos)
        assert torch.equal(out, one.expand_as(out))
        qk_norm_rope_backward(one, None, x, None, None, None, cos, sin, one, None, positions=pos[:1])
        qk_norm_rope_backward(out, None, many, None, None, None, cos, sin, out, None, positions=pos)
        assert torch.equal(out, one.expand_as(out))


def test_two_host_threads():
    import threading
    cos, sin, _, _ = _angles(64, 500)
    g = draw((64,), 80, 0.1, 1.0).to(DEV)
    sets, bad = [], []
    for i in range(2):
        x = draw((1, 400 + 90 * i, 4 + i, 64), 81 + i).to(DEV)
        o = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(g)]
        qk_norm_rope(x, None, g, None, cos, sin, o[0], None, positions=torch.arange(x.shape[1], device=DEV) % 90)
        qk_norm_rope_backward(x, None, x, None, g, None, cos, sin, o[1], None, dgamma_q=o[2])
        sets.append((x, o, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(x, want, stream):
        try:
            pos = torch.arange(x.shape[1], device=DEV) % 90
            outs = [[torch.empty_like(t) for t in want] for _ in range(20)]
            torch.cuda.synchronize()
            for o in outs:
                qk_norm_rope(x, None, g, None, cos, sin, o[0], None, positions=pos, stream=stream)
                qk_norm_rope_backward(x, None, x, None, g, None, cos, sin, o[1], None, dgamma_q=o[2], stream=stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for o in outs for a, b in zip(o, want)):
                bad.append("outputs differ")
        except Exception as e:  # noqa: BLE001 - reported by the test
            bad.append(repr(e))

    ts = [threading.Thread(target=work, args=s) for s in sets]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def test_no_tokens():
    q, k = torch.empty(2, 0, 4, 32, device=DEV), torch.empty(2, 0, 1, 32, device=DEV)
    g = torch.ones(32, device=DEV)
    cos, sin, _, _ = _angles(32)
    qk_norm_rope(q, k, g, g, cos, sin, q.clone(), k.clone())
    for dt in DTYPES.values():
        d1, d2 = torch.full((32,), 5.0, dtype=dt, device=DEV), torch.full((32,), 5.0, dtype=dt, device=DEV)
        qk_norm_rope_backward(q.clone(), k.clone(), q, k, g.to(dt), None, cos, sin, q.clone(), k.clone(), dgamma_q=d1,
                              dgamma_k=d2)
        assert not d1.any() and not d2.any()


def test_gradient_against_differences():
    b, t, h, dim, rot = 1, 6, 2, 20, 12
    q = draw((b, t, h, dim), 21).to(DEV)
    g, dy = draw((dim,), 22, 0.2, 1.0).to(DEV), draw((b, t, h, dim), 23).to(DEV)
    cos, sin, cn, sn = _angles(rot)
    c, s = R.token_angles(cn, sn, rot, b, t)
    for inter in (False, True):
        dx, dg = torch.empty_like(q), torch.empty_like(g)
        qk_norm_rope_backward(dy, None, q, None, g, None, cos, sin, dx, None, dgamma_q=dg, interleaved=inter, eps=EPS)
        f = lambda x, gm: (R.qk_norm_rope(x, gm, c, s, rot, inter, EPS) * h64(dy)).sum()
        v, w = h64(draw((b, t, h, dim), 24)), h64(draw((dim,), 25))
        num = (f(h64(q) + 1e-5 * v, h64(g) + 1e-5 * w) - f(h64(q) - 1e-5 * v, h64(g) - 1e-5 * w)) / 2e-5
        got = (h64(dx) * v).sum() + (h64(dg) * w).sum()
        assert abs(got - num) <= 1e-7 + 4 * K * U * (np.abs(h64(dy)).sum() * 4)


def test_workspaces_and_repeats():
    q, k = draw((1, 900, 8, 64), 31).to(DEV), draw((1, 900, 2, 64), 32).to(DEV)
    g = torch.ones(64, device=DEV)
    cos, sin, _, _ = _angles(64, 900)
    outs = []
    ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for w in (None, ws, ws):
        o = [torch.empty_like(v) for v in (q, k, g, g)]
        qk_norm_rope_backward(q, k, q, k, g, g, cos, sin, o[0], o[1], dgamma_q=o[2], dgamma_k=o[3], workspace=w)
        outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    with pytest.raises(MuonError) as e:
        qk_norm_rope_backward(q, k, q, k, g, g, cos, sin, o[0], o[1], dgamma_q=o[2], workspace=ws[:64])
    assert e.value.status == 5
    # one of the two gains alone has the same bits
    d = torch.empty_like(g)
    qk_norm_rope_backward(q, k, q, k, g, g, cos, sin, o[0], o[1], dgamma_k=d)
    assert torch.equal(d, outs[0][3])


def test_graph_replays_and_streams():
    xs = [draw((2, 300, 6, 64), 41 + i).to(DEV).bfloat16() for i in range(3)]
    q = xs[0].clone()
    g = draw((64,), 45, 0.1, 1.0).to(DEV)
    cos, sin, _, _ = _angles(64, 400)
    pos = torch.arange(300, device=DEV)
    new = lambda: [torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(g)]

    def step(x, o, stream=None):
        qk_norm_rope(x, None, g, None, cos, sin, o[0], None, positions=pos, stream=stream)
        qk_norm_rope_backward(o[0], None, x, None, g, None, cos, sin, o[1], None, dgamma_q=o[2], positions=pos,
                              stream=stream)

    rec = new()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(q, rec)
    side = torch.cuda.Stream()
    for x in xs + xs:
        q.copy_(x)
        pos.add_(7)
        graph.replay()
        torch.cuda.synchronize()
        o = new()
        torch.cuda.synchronize()
        step(x, o, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, rec))
