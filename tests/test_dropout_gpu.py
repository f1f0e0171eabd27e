"""GPU dropout against the generator's definition: the mask bit for bit, the
values to the rounding of the stored type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import dropout
from oracle import ops_ref as R
from tests.ops_helpers import DEV, DTYPES, U, draw, h64, half_step, within

pytestmark = pytest.mark.gpu


def _check(out, x, res, p, seed, offset):
    xs = h64(x)
    rs = None if res is None else h64(res)
    want = R.dropout(xs, p, seed, offset, rs)
    mag = np.abs(want) if rs is None else np.abs(want) + np.abs(rs)
    # one fused multiply-add in fp32 with the scale rounded to fp32, then one rounding
    within(out, want, half_step(x.dtype) * np.abs(want) * (1 + 1e-6) + 4 * U * mag, "out")
    if res is None:
        keep = R.keep_mask(*xs.shape, p, seed, offset)
        assert np.array_equal(h64(out) != 0, keep & (xs != 0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 9), (1, 100003), (1000, 3), (70001, 17), (257, 1537),
                                       (64, 4096)])
def test_matches_the_definition(rows, cols, dt):
    x = draw((rows, cols), rows + cols, 1.0, 0.5, DTYPES[dt]).to(DEV)
    res = draw((rows, cols), 2, 2.0, 0.0, DTYPES[dt]).to(DEV)
    for p, seed, offset in ((0.1, 1, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1), (0.9, 1 << 40, 1 << 32)):
        out = torch.empty_like(x)
        dropout(x, out, p=p, seed=seed, offset=offset)
        _check(out, x, None, p, seed, offset)
        dropout(x, out, p=p, seed=seed, offset=offset, residual=res)
        _check(out, x, res, p, seed, offset)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ends_of_p(dt):
    x = draw((40, 333), 5, dtype=DTYPES[dt]).to(DEV)
    res = draw((40, 333), 6, dtype=DTYPES[dt]).to(DEV)
    out = torch.empty_like(x)
    dropout(x, out, p=0.0, seed=3)
    assert torch.equal(out, x)
    dropout(x, out, p=1.0, seed=3)
    assert not out.any()
    dropout(x, out, p=1.0, seed=3, residual=res)
    assert torch.equal(out, res)
    dropout(x, out, p=2.0 ** -18, seed=3)  # nearer to 0 than to the first step
    assert torch.equal(out, x)


def test_dropped_elements_are_zero_whatever_they_hold():
    x = torch.full((50, 77), float("nan"), device=DEV)
    x[::2] = float("inf")
    out = torch.empty_like(x)
    dropout(x, out, p=0.5, seed=11)
    keep = torch.from_numpy(R.keep_mask(50, 77, 0.5, 11, 0)).to(DEV)
    assert (out[~keep] == 0).all() and not torch.isfinite(out[keep]).any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_place_strides_and_gaps(dt):
    rows, cols, ld = 61, 203, 210
    x = draw((rows, cols), 21, dtype=DTYPES[dt]).to(DEV)
    res = draw((rows, cols), 22, dtype=DTYPES[dt]).to(DEV)
    want, wres = torch.empty_like(x), torch.empty_like(x)
    dropout(x, want, p=0.3, seed=4, offset=9)
    dropout(x, wres, p=0.3, seed=4, offset=9, residual=res)
    buf = torch.full((rows * ld + 3,), 9.0, dtype=DTYPES[dt], device=DEV)
    v = buf[3:].view(rows, ld)[:, :cols]
    v.copy_(x)
    dropout(v, v, p=0.3, seed=4, offset=9)
    assert torch.equal(v, want)
    v.fill_(9.0)
    assert (buf == 9.0).all()
    r2 = res.clone()
    dropout(x, r2, p=0.3, seed=4, offset=9, residual=r2)
    assert torch.equal(r2, wres)
    x2 = x.clone()   # all three the same tensor
    dropout(x2, x2, p=0.3, seed=4, offset=9, residual=x2)
    self_res = torch.empty_like(x)
    dropout(x, self_res, p=0.3, seed=4, offset=9, residual=x)
    assert torch.equal(x2, self_res)
    x3 = x.view(61, 7, 29)   # rows are what precedes the last dimension
    o3 = torch.empty_like(x3)
    dropout(x3, o3, p=0.3, seed=4, offset=9)
    flat = torch.empty(61 * 7, 29, dtype=DTYPES[dt], device=DEV)
    dropout(x.view(61 * 7, 29), flat, p=0.3, seed=4, offset=9)
    assert torch.equal(o3.view(61 * 7, 29), flat)


def test_offsets_past_32_bits():
    """Rows that lie further apart than 2^32 elements, and one row longer than
    2^32 elements, whose ends are checked."""
    ld = (1 << 32) + 24
    buf = torch.zeros(2 * ld, dtype=torch.bfloat16, device=DEV)
    x = buf.view(2, ld)[:, 16:1040]
    x.copy_(draw((2, 1024), 31, dtype=torch.bfloat16))
    out = torch.empty(2, 1024, dtype=torch.bfloat16, device=DEV)
    dropout(x, out, p=0.4, seed=8, offset=2)
    _check(out, x.contiguous(), None, 0.4, 8, 2)
    n = (1 << 32) + 41
    row = buf[:n].fill_(1.0)
    dropout(row, row, p=0.25, seed=77, offset=1)
    t = R.threshold(0.25)
    for at in (0, (1 << 32) - 64, n - 57):
        at = at // 8 * 8
        m = min(64, n - at)
        block = np.arange(at // 8, (at + m + 7) // 8, dtype=np.uint64)
        w = R.philox([block, np.uint64(0), np.uint64(1), np.uint64(0)], [77, 0])
        u = np.stack([np.stack([v & np.uint64(0xFFFF), v >> np.uint64(16)], -1) for v in w], -2).reshape(-1)[:m]
        assert np.array_equal(row[at:at + m].cpu().float().numpy() != 0, u >= t), at
    # 2^32 draws of rate 3/4, counted in slices: 6 standard deviations are 4e-5
    kept = sum(int((row[i:i + (1 << 28)] != 0).sum()) for i in range(0, n, 1 << 28))
    assert abs(kept / n - 0.75) < 5e-5


def test_gradient_is_the_same_call():
    """d(sum(out * w)) / dx = dropout(w): the mask does not depend on x."""
    x, w = draw((33, 130), 41).to(DEV), draw((33, 130), 42).to(DEV)
    kw = dict(p=0.2, seed=5, offset=6)
    dx = torch.empty_like(x)
    dropout(w, dx, **kw)
    v = h64(draw((33, 130), 43))
    f = lambda z: (R.dropout(z, 0.2, 5, 6) * h64(w)).sum()
    d = (f(h64(x) + v) - f(h64(x) - v)) / 2
    assert abs((h64(dx) * v).sum() - d) <= 8 * U * np.abs(h64(dx) * v).sum() + 1e-11


def test_device_offset_streams_and_determinism():
    x = draw((500, 900), 51, dtype=torch.bfloat16).to(DEV)
    a, b, c = (torch.empty_like(x) for _ in range(3))
    dropout(x, a, p=0.1, seed=9, offset=(1 << 32) + 12)
    word = torch.full((1,), (1 << 32) + 2, dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()
    dropout(x, b, p=0.1, seed=9, offset=10, offset_dev=word, stream=torch.cuda.Stream())
    dropout(x, c, p=0.1, seed=9, offset=(1 << 64) - 1, offset_dev=word + 11)  # modulo 2^64
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
