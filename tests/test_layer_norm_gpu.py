"""GPU layer norm (forward, backward, alone and fused with dropout and the
residual add) against the fp64 oracle, at every boundary of the kernels' row
splits, and the properties the header states."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import (dropout, dropout_add_layer_norm, dropout_add_layer_norm_backward, layer_norm,
                                  layer_norm_backward)
from newton_schulz_05_amd import MuonError
from oracle import ops_ref as R
from tests.ops_helpers import DEV, DTYPES, K, U, draw, h64, half_step, norm_bounds, norm_grad_bounds, within

pytestmark = pytest.mark.gpu
EPS = 1e-5
# around each change of the number of threads or vectors a row takes
WIDTHS = [1, 2, 7, 8, 9, 63, 65, 127, 128, 129, 255, 257, 511, 513, 1023, 1024, 1025, 2047, 2049, 4096, 4097, 6145, 8191,
          8193, 10241, 12289, 16384, 16385, 20481, 32761, 32768]
KINDS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]


def _inputs(rows, cols, dt, wdt, seed, mean=0.3):
    x = draw((rows, cols), seed, 1.0, mean, DTYPES[dt]).to(DEV)
    gamma = draw((cols,), seed + 1, 0.2, 1.0, DTYPES[wdt]).to(DEV)
    beta = draw((cols,), seed + 2, 0.2, 0.0, DTYPES[wdt]).to(DEV)
    return x, gamma, beta


def _forward(x, gamma, beta, **kw):
    rows = x.shape[0]
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(rows, device=DEV) for _ in range(2))
    layer_norm(x, gamma, beta, y, mean=mean, rstd=rstd, eps=EPS, **kw)
    return y, mean, rstd


def _check_forward(x, gamma, beta, got):
    y, mean, rstd = got
    xs = h64(x)
    g, b = (None if t is None else h64(t) for t in (gamma, beta))
    wy, wm, wr = R.layer_norm(xs, g, b, EPS)
    by, bm, br = norm_bounds(xs, g, b, wy, wm, wr, x.dtype)
    within(mean, wm, bm, "mean")
    within(rstd, wr, br, "rstd")
    within(y, wy, by, "y")


def _chain(rows):
    return -(-rows // 256) + 8  # rows of one thread, at the fewest threads a column has


def _check_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, extra=None):
    d, xs, m, r = h64(dy), h64(x), h64(mean), h64(rstd)
    g = None if gamma is None else h64(gamma)
    wx, wg, wb = R.layer_norm_backward(d, xs, g, m, r)
    if extra is not None:
        wx = wx + h64(extra)
    wdt = (dgamma if dgamma is not None else dx).dtype
    bx, sg, sb, chain, half = norm_grad_bounds(d, xs, g, m, r, wx, dx.dtype, wdt, _chain(x.shape[0]))
    if extra is not None:
        bx = bx + 2 * U * np.abs(h64(extra))
    within(dx, wx, bx, "dx")
    if dgamma is not None:
        within(dgamma, wg, half * np.abs(wg) * (1 + 1e-6) + chain * sg, "dgamma")
    if dbeta is not None:
        within(dbeta, wb, half * np.abs(wb) * (1 + 1e-6) + chain * sb, "dbeta")
    return wx, bx


@pytest.mark.parametrize("dt,wdt", KINDS)
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_and_backward_match_the_oracle(cols, dt, wdt):
    for rows in (1, 5, 67):
        x, gamma, beta = _inputs(rows, cols, dt, wdt, 100 + cols + rows)
        got = _forward(x, gamma, beta)
        _check_forward(x, gamma, beta, got)
        dy = draw((rows, cols), 7 + cols, 0.1, 0.02, DTYPES[dt]).to(DEV)
        dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
        layer_norm_backward(dy, x, gamma, got[1], got[2], dx, dgamma=dg, dbeta=db)
        _check_backward(dy, x, gamma, got[1], got[2], dx, dg, db)


@pytest.mark.parametrize("dt,wdt", KINDS[:3])
@pytest.mark.parametrize("rows,cols", [(5000, 24), (4099, 640), (1031, 1536), (1025, 4096), (530, 8192), (257, 40),
                                       (300, 400), (700, 1000), (400, 9000), (300, 12300), (300, 17001), (300, 21000),
                                       (270, 30000), (9000, 200), (3000, 250)])
def test_many_rows(rows, cols, dt, wdt):
    """More rows than workgroups: each keeps several, and the partial sums of
    dgamma and dbeta are joined by the second kernel."""
    x, gamma, beta = _inputs(rows, cols, dt, wdt, rows)
    got = _forward(x, gamma, beta)
    _check_forward(x, gamma, beta, got)
    dy = draw((rows, cols), 8 + cols, 0.1, 0.02, DTYPES[dt]).to(DEV)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    layer_norm_backward(dy, x, gamma, got[1], got[2], dx, dgamma=dg, dbeta=db)
    _check_backward(dy, x, gamma, got[1], got[2], dx, dg, db)
    again = [torch.empty_like(t) for t in (dx, dg, db)]
    layer_norm_backward(dy, x, gamma, got[1], got[2], again[0], dgamma=again[1], dbeta=again[2])
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dg, db)))


def test_gradient_against_differences():
    """<gradient, v> of the GPU against the central difference of the oracle's
    forward pass in fp64 along v."""
    rows, cols = 9, 133
    x, gamma, beta = _inputs(rows, cols, "f32", "f32", 31)
    _, mean, rstd = _forward(x, gamma, beta)
    dy = draw((rows, cols), 32).to(DEV)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db)
    args = [h64(x), h64(gamma), h64(beta)]
    for i, grad in enumerate((dx, dg, db)):
        v = h64(draw(tuple(grad.shape), 33 + i))
        h = 1e-5
        side = []
        for s in (h, -h):
            a = list(args)
            a[i] = a[i] + s * v
            side.append((R.layer_norm(*a, EPS)[0] * h64(dy)).sum())
        want = (side[0] - side[1]) / (2 * h)
        # fp32 sums of |gradient * v|, mean and rstd themselves in fp32
        assert abs((h64(grad) * v).sum() - want) <= 1e-7 + 4 * K * U * np.abs(h64(grad) * v).sum()


@pytest.mark.parametrize("which", ["none", "gamma", "beta"])
def test_optional_arguments(which):
    x, gamma, beta = _inputs(21, 300, "bf16", "f32", 41)
    g, b = (gamma if which == "gamma" else None), (beta if which == "beta" else None)
    got = _forward(x, g, b)
    _check_forward(x, g, b, got)
    y = torch.empty_like(x)
    layer_norm(x, g, b, y, eps=EPS)              # no statistics: serving
    assert torch.equal(y, got[0])
    dy = draw((21, 300), 42, 0.1, 0.0, torch.bfloat16).to(DEV)
    full = [torch.empty_like(x), torch.empty(300, device=DEV), torch.empty(300, device=DEV)]
    layer_norm_backward(dy, x, g, got[1], got[2], full[0], dgamma=full[1], dbeta=full[2])
    _check_backward(dy, x, g, got[1], got[2], *full)
    for want in ((False, False), (True, False), (False, True)):
        dx = torch.empty_like(x)
        dg, db = (torch.empty(300, device=DEV) if w else None for w in want)
        layer_norm_backward(dy, x, g, got[1], got[2], dx, dgamma=dg, dbeta=db)
        assert torch.equal(dx, full[0])
        assert dg is None or torch.equal(dg, full[1])
        assert db is None or torch.equal(db, full[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 136, 1537, 9001])
def test_strides_and_alignment_change_no_bit(dt, cols):
    """Rows that are slices of a wider, oddly placed buffer give the same bits
    as dense ones, and what lies between them stays as it was."""
    rows, ld = 37, cols + 3
    x, gamma, beta = _inputs(rows, cols, dt, dt, 51)
    dy = draw((rows, cols), 52, 0.1, 0.0, DTYPES[dt]).to(DEV)

    def slot(t=None, shift=1):
        buf = torch.full((rows * ld + 8,), 7.0, dtype=DTYPES[dt], device=DEV)
        v = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
        if t is not None:
            v.copy_(t)
        return buf, v

    y, mean, rstd = _forward(x, gamma, beta)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db)
    (_, xv), (_, dv), (yb, yv), (xb, dxv) = slot(x, 1), slot(dy, 3), slot(shift=5), slot(shift=2)
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    layer_norm(xv, gamma, beta, yv, mean=m2, rstd=r2, eps=EPS)
    dg2, db2 = torch.empty_like(gamma), torch.empty_like(gamma)
    layer_norm_backward(dv, xv, gamma, m2, r2, dxv, dgamma=dg2, dbeta=db2)
    for a, b in ((y, yv), (mean, m2), (rstd, r2), (dx, dxv), (dg, dg2), (db, db2)):
        assert torch.equal(a, b)
    for buf, v, shift in ((yb, yv, 5), (xb, dxv, 2)):
        v.fill_(7.0)
        assert (buf == 7.0).all(), "bytes outside the rows were written"
    # two column slices of one buffer, input and output
    wide = torch.zeros(rows, 2 * cols, dtype=DTYPES[dt], device=DEV)
    wide[:, :cols] = x
    layer_norm(wide[:, :cols], gamma, beta, wide[:, cols:], eps=EPS)
    assert torch.equal(wide[:, cols:], y) and torch.equal(wide[:, :cols], x)


def test_offsets_past_32_bits():
    ld = (1 << 32) + 16
    buf = torch.empty(2 * ld, dtype=torch.bfloat16, device=DEV)
    x = buf.view(2, ld)[:, 8:520]
    x.copy_(draw((2, 512), 61, 1.0, 0.2, torch.bfloat16))
    dense = x.contiguous()
    y, mean, rstd = _forward(dense, None, None)
    out = buf.view(2, ld)[:, 1000:1512]
    layer_norm(x, None, None, out, eps=EPS)
    assert torch.equal(out, y)
    dx = torch.empty_like(dense)
    layer_norm_backward(out, x, None, mean, rstd, dx)
    want = torch.empty_like(dense)
    layer_norm_backward(y, dense, None, mean, rstd, want)
    assert torch.equal(dx, want)


@pytest.mark.parametrize("rows,cols", [((1 << 25) + 77, 5), ((1 << 21) + 3, 1030)])
def test_more_rows_than_a_launch_has_workgroups(rows, cols):
    """The forward launch is capped and loops: the last rows come out as they
    do alone."""
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).fill_(1.0)
    tail = 700
    x[-tail:] = draw((tail, cols), 63, 1.0, 0.2, torch.bfloat16).to(DEV)
    gamma = draw((cols,), 64, 0.2, 1.0).to(DEV)
    y, mean, rstd = _forward(x, gamma, None)
    want = _forward(x[-tail:].clone(), gamma, None)
    for a, b in zip((y, mean, rstd), want):
        assert torch.equal(a[-tail:], b)
    assert not y[:-tail].any() and (mean[:-tail] == 1.0).all()


def test_parameters_at_odd_addresses():
    """gamma, beta and their gradients as slices of a flat parameter buffer."""
    for rows in (9, 400):
        x, gamma, beta = _inputs(rows, 77, "bf16", "bf16", 65)
        dy = draw((rows, 77), 66, 0.1, 0.0, torch.bfloat16).to(DEV)
        flat = torch.zeros(2 * 77 + 3, dtype=torch.bfloat16, device=DEV)
        gv, bv = flat[1:78], flat[79:156]
        gv.copy_(gamma)
        bv.copy_(beta)
        y, mean, rstd = _forward(x, gamma, beta)
        y2, _, _ = _forward(x, gv, bv)
        assert torch.equal(y, y2)
        grads = torch.full_like(flat, 3.0)
        dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
        layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db)
        layer_norm_backward(dy, x, gv, mean, rstd, dx, dgamma=grads[1:78], dbeta=grads[79:156])
        assert torch.equal(grads[1:78], dg) and torch.equal(grads[79:156], db)
        assert (grads[[0, 78, 156]] == 3.0).all()


def test_leading_dimensions():
    x, gamma, beta = _inputs(24, 96, "bf16", "bf16", 71)
    y, mean, rstd = _forward(x, gamma, beta)
    x3 = x.view(4, 6, 96)
    y3, m3 = torch.empty_like(x3), torch.empty(4, 6, device=DEV)
    layer_norm(x3, gamma, beta, y3, mean=m3, eps=EPS)
    assert torch.equal(y3.view(24, 96), y) and torch.equal(m3.view(-1), mean)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_hard_rows(dt):
    """A large common offset (a one-pass variance would cancel), constant
    rows, rows of one spike, tiny and huge values."""
    cols = 1000
    x = draw((8, cols), 81, 1.0, 0.0, DTYPES[dt])
    x[1] = x[1] + 512
    x[2] = 3.0
    x[3] = 0.0
    x[4] = 0.0
    x[4, 77] = 100.0
    x[5] = x[5] * 1e-18
    x[6] = x[6] * 1e15
    x = x.to(DEV)
    got = _forward(x, None, None)
    _check_forward(x, None, None, got)
    assert (h64(got[0])[3] == 0).all()
    dy = draw((8, cols), 82, 1.0, 0.0, DTYPES[dt]).to(DEV)
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    layer_norm_backward(dy, x, None, got[1], got[2], dx, dgamma=dg, dbeta=db)
    _check_backward(dy, x, None, got[1], got[2], dx, dg, db)


def test_a_bad_row_stays_alone():
    x, gamma, beta = _inputs(70, 513, "f32", "f32", 91)
    clean = _forward(x, gamma, beta)
    x2 = x.clone()
    x2[3, 5], x2[40, 500], x2[69, 512] = float("nan"), float("inf"), float("-inf")
    got = _forward(x2, gamma, beta)
    ok = torch.ones(70, dtype=torch.bool)
    ok[[3, 40, 69]] = False
    assert torch.equal(got[0].cpu()[ok], clean[0].cpu()[ok])
    assert torch.isnan(got[0][3]).all() and torch.isnan(got[0][40]).any()
    dy = draw((70, 513), 92).to(DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    layer_norm_backward(dy, x, gamma, clean[1], clean[2], a)
    layer_norm_backward(dy, x2, gamma, got[1], got[2], b)
    assert torch.equal(a.cpu()[ok], b.cpu()[ok])


def test_no_rows():
    gamma = torch.ones(50, device=DEV)
    e = torch.empty(0, 50, device=DEV)
    layer_norm(e, gamma, None, torch.empty_like(e))
    dg, db = torch.full_like(gamma, 5.0), torch.full_like(gamma, 5.0)
    st = torch.empty(0, device=DEV)
    layer_norm_backward(e, e, gamma, st, st, torch.empty_like(e), dgamma=dg, dbeta=db)
    assert not dg.any() and not db.any()
    dropout(e, e, p=0.5, seed=1)
    dropout_add_layer_norm(e, e, gamma, None, torch.empty_like(e), torch.empty_like(e), p=0.5, seed=1)
    dg.fill_(5.0)
    dropout_add_layer_norm_backward(e, e, gamma, st, st, torch.empty_like(e), torch.empty_like(e), p=0.5, seed=1,
                                    dgamma=dg)
    assert not dg.any()


# ---- fused with dropout and the residual add ------------------------------------------

RNG = dict(p=0.2, seed=0x1234567890ABCDEF, offset=(1 << 33) + 5)


@pytest.mark.parametrize("dt,wdt", KINDS)
@pytest.mark.parametrize("cols", [1, 7, 8, 121, 129, 520, 1024, 1543, 4096, 8193, 16390, 32768])
def test_fused_forward_is_the_two_calls(cols, dt, wdt):
    rows = 19
    x, gamma, beta = _inputs(rows, cols, dt, wdt, 300 + cols)
    res = draw((rows, cols), 301, 2.0, 0.0, DTYPES[dt]).to(DEV)
    h0 = torch.empty_like(x)
    dropout(x, h0, residual=res, **RNG)
    y0, m0, r0 = _forward(h0, gamma, beta)
    h, y = torch.empty_like(x), torch.empty_like(x)
    m, r = torch.empty_like(m0), torch.empty_like(r0)
    dropout_add_layer_norm(x, res, gamma, beta, h, y, mean=m, rstd=r, eps=EPS, **RNG)
    for a, b in ((h, h0), (y, y0), (m, m0), (r, r0)):
        assert torch.equal(a, b)
    inplace = res.clone()
    dropout_add_layer_norm(x, inplace, gamma, beta, inplace, y.zero_(), eps=EPS, **RNG)
    assert torch.equal(inplace, h0) and torch.equal(y, y0)


@pytest.mark.parametrize("dt,wdt", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 8), (19, 1), (19, 121), (700, 129), (45, 1543), (600, 4096), (33, 8193),
                                       (9, 16390), (7, 32768), (260, 100), (400, 9000), (300, 12300),
                                       (300, 17001), (270, 21000), (270, 30000), (9000, 200)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_fused_backward(rows, cols, dt, wdt, with_dh):
    h, gamma, _ = _inputs(rows, cols, dt, wdt, 400 + cols)
    _, mean, rstd = _forward(h, gamma, None)
    dy = draw((rows, cols), 401, 0.1, 0.01, DTYPES[dt]).to(DEV)
    dh = draw((rows, cols), 402, 0.1, 0.0, DTYPES[dt]).to(DEV) if with_dh else None
    dx, dres = torch.empty_like(h), torch.empty_like(h)
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    dropout_add_layer_norm_backward(dy, h, gamma, mean, rstd, dx, dres, dh=dh, dgamma=dg, dbeta=db, **RNG)
    want, bound = _check_backward(dy, h, gamma, mean, rstd, dres, dg, db, extra=dh)
    keep = R.keep_mask(rows, cols, RNG["p"], RNG["seed"], RNG["offset"])
    scale = 65536 / (65536 - R.threshold(RNG["p"]))
    within(dx, np.where(keep, want * scale, 0.0), np.where(keep, scale * bound + 4 * U * np.abs(want), 0.0), "dx")
    # the norm's own backward gives the same sums
    dg2, db2, dx2 = torch.empty_like(gamma), torch.empty_like(gamma), torch.empty_like(h)
    layer_norm_backward(dy, h, gamma, mean, rstd, dx2, dgamma=dg2, dbeta=db2)
    assert torch.equal(dg, dg2) and torch.equal(db, db2)
    if not with_dh:
        assert torch.equal(dres, dx2)


# ---- streams and graphs ----------------------------------------------------------------

def test_side_stream_and_workspace():
    rows, cols = 900, 1200
    x, gamma, beta = _inputs(rows, cols, "bf16", "f32", 501)
    dy = draw((rows, cols), 502, 0.1, 0.0, torch.bfloat16).to(DEV)
    y, mean, rstd = _forward(x, gamma, beta)
    want = [torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)]
    layer_norm_backward(dy, x, gamma, mean, rstd, want[0], dgamma=want[1], dbeta=want[2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(3):  # several calls in flight on two streams, each with a workspace of its own
        for st in (side, None):
            o = [torch.empty_like(t) for t in want]
            layer_norm_backward(dy, x, gamma, mean, rstd, o[0], dgamma=o[1], dbeta=o[2], stream=st)
            outs.append(o)
    torch.cuda.synchronize()
    ws = torch.full((1 << 23,), 0xFF, dtype=torch.uint8, device=DEV)  # needs no clearing
    o = [torch.empty_like(t) for t in want]
    layer_norm_backward(dy, x, gamma, mean, rstd, o[0], dgamma=o[1], dbeta=o[2], workspace=ws)
    outs.append(o)
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    with pytest.raises(MuonError) as e:
        layer_norm_backward(dy, x, gamma, mean, rstd, o[0], dgamma=o[1], dbeta=o[2], workspace=ws[:64])
    assert e.value.status == 5


def test_graph_replays_draw_new_masks():
    """A fused forward and backward recorded once: every replay takes the mask
    of the device offset at that time and gives the eager call's bits."""
    rows, cols = 300, 2056
    x, gamma, beta = _inputs(rows, cols, "bf16", "bf16", 511)
    res = draw((rows, cols), 512, 1.0, 0.0, torch.bfloat16).to(DEV)
    dy = draw((rows, cols), 513, 0.1, 0.0, torch.bfloat16).to(DEV)
    word = torch.zeros(1, dtype=torch.int64, device=DEV)

    def outputs():
        return dict(h=torch.zeros_like(x), y=torch.zeros_like(x), mean=torch.zeros(rows, device=DEV),
                    rstd=torch.zeros(rows, device=DEV), dx=torch.zeros_like(x), dres=torch.zeros_like(x),
                    dgamma=torch.zeros_like(gamma), dbeta=torch.zeros_like(gamma))

    def step(o, offset, dev):
        rng = dict(p=0.3, seed=99, offset=offset, offset_dev=dev)
        dropout_add_layer_norm(x, res, gamma, beta, o["h"], o["y"], mean=o["mean"], rstd=o["rstd"], eps=EPS, **rng)
        dropout_add_layer_norm_backward(dy, o["h"], gamma, o["mean"], o["rstd"], o["dx"], o["dres"],
                                        dgamma=o["dgamma"], dbeta=o["dbeta"], **rng)

    rec = outputs()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(rec, 17, word)
    torch.cuda.synchronize()
    assert not rec["y"].any()
    seen = []
    for i in (0, 1, 2, (1 << 40) + 3):
        word.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        eager = outputs()
        step(eager, 17 + i, None)
        torch.cuda.synchronize()
        for n in rec:
            assert torch.equal(rec[n], eager[n]), (i, n)
        seen.append(rec["h"].clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_two_graphs_share_a_workspace():
    shapes = [(700, 1030), (350, 4096)]
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    sets = []
    for i, (rows, cols) in enumerate(shapes):
        x, gamma, beta = _inputs(rows, cols, "f32", "f32", 520 + i)
        _, mean, rstd = _forward(x, gamma, beta)
        dy = draw((rows, cols), 530 + i).to(DEV)
        want = [torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)]
        layer_norm_backward(dy, x, gamma, mean, rstd, want[0], dgamma=want[1], dbeta=want[2])
        got = [torch.zeros_like(t) for t in want]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            layer_norm_backward(dy, x, gamma, mean, rstd, got[0], dgamma=got[1], dbeta=got[2], workspace=ws)
        sets.append((g, got, want, (x, gamma, mean, rstd, dy)))  # the graph reads them on each replay
    for _ in range(3):
        for g, got, want, _ in sets:
            for t in got:
                t.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in sets:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
