"""Binding of the training operators beside the step (include/muon.h): layer
norm, dropout, the two fused with the residual add, and the expert router.

Argument marshalling only, like ``binding``: the caller gives the output
tensors, every call is one C call on the current stream of the tensors'
device (or on ``stream``), and nothing is kept between calls.  A matrix
argument is any tensor whose last dimension is contiguous and whose leading
dimensions lie one row stride apart (a column slice of a wider buffer, a
[batch, time, cols] activation).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from .binding import MUON_BF16, MUON_F32, MuonError, _check, load_library


_CODES = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}


def _dtype_code(dt: torch.dtype) -> int:
    code = _CODES.get(dt)
    if code is None:
        raise MuonError(3, f"unsupported dtype {dt}")
    return code


def _matrix(t: torch.Tensor, what: str) -> Tuple[int, int, int]:
    """(rows, cols, row stride) of a matrix argument."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        rows, cols = shape
        ld, step = stride
        if step != 1 and cols > 1:
            raise MuonError(1, f"{what}: the last dimension is not contiguous")
        return rows, cols, ld if rows > 1 else cols
    if not shape:
        raise MuonError(2, f"{what} needs at least one dimension")
    cols = shape[-1]
    if stride[-1] != 1 and cols > 1:
        raise MuonError(1, f"{what}: the last dimension is not contiguous")
    rows, ld = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 0:
            return 0, cols, cols
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise MuonError(1, f"{what}: the rows do not lie one stride apart")
        rows *= n
    return rows, cols, cols if ld is None else ld


def _same(t: torch.Tensor, like: torch.Tensor, what: str) -> int:
    """Row stride of a matrix that has to match `like`."""
    shape = t.shape
    if shape != like.shape:
        raise MuonError(2, f"{what} has shape {tuple(shape)}, expected {tuple(like.shape)}")
    if t.dtype is not like.dtype:
        raise MuonError(3, f"{what} has dtype {t.dtype}, expected {like.dtype}")
    stride = t.stride()
    if len(shape) == 2 and stride[1] == 1:
        return stride[0] if shape[0] > 1 else shape[1]
    return _matrix(t, what)[2]


def _flat(t: Optional[torch.Tensor], n: int, dtypes, what: str) -> Optional[int]:
    """Pointer of a contiguous argument of n elements, or None."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise MuonError(3, f"{what} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.numel() != n:
        raise MuonError(2, f"{what} has {t.numel()} elements, expected {n}")
    if not t.is_contiguous():
        raise MuonError(1, f"{what} is not contiguous")
    return t.data_ptr()


_F32, _I32, _MASK, _WORD = (torch.float32,), (torch.int32,), (torch.uint8, torch.bool), (torch.int64,)


def _device(stream, *tensors) -> Tuple[int, int]:
    """(device index, stream handle) of a call: that of its tensors, which must
    share one, and their device's current stream unless one is given.  The
    handle is read without making a Stream object, which would cost as much
    as the launch (2.7 us of 9.7 for a one-row layer_norm)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise MuonError(1, "every tensor must be a device tensor")
            if dev is not None:
                raise MuonError(1, f"tensors on devices {dev} and {d}")
            dev = d
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise MuonError(1, f"a stream of {stream.device} for tensors on device {dev}")
    return dev, stream.cuda_stream


def _call(dev: int, f, *args) -> None:
    """The C call with the tensors' device current."""
    if torch._C._cuda_getDevice() == dev:
        _check(f(*args))
    else:
        with torch.cuda.device(dev):
            _check(f(*args))


def _workspace(given: Optional[torch.Tensor], need: int, stream, dev: int, handle: int):
    """(tensor, pointer, bytes): the caller's workspace, or one from torch's
    allocator that belongs to the call's stream."""
    if given is not None:
        if not given.is_contiguous():
            raise MuonError(5, "workspace is not contiguous")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    if stream is None or handle == torch._C._cuda_getCurrentRawStream(dev):
        t = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(need, dtype=torch.uint8, device=dev)
    return t, t.data_ptr(), need


def _param(t: Optional[torch.Tensor], dt: torch.dtype, cols: int, what: str) -> Optional[int]:
    """Pointer of a 1-D parameter or its gradient, or None."""
    if t is None:
        return None
    if t.dtype is not dt:
        raise MuonError(3, f"{what} has dtype {t.dtype}, expected {dt}")
    if t.numel() != cols:
        raise MuonError(2, f"{what} has {t.numel()} elements, expected {cols}")
    if not t.is_contiguous():
        raise MuonError(1, f"{what} is not contiguous")
    return t.data_ptr()


def _param_dtype(x: torch.Tensor, *params) -> torch.dtype:
    """The parameters' common dtype: that of the first one given."""
    for t in params:
        if t is not None:
            return t.dtype
    return x.dtype


def _u64(v: int, what: str) -> int:
    if type(v) is not int:
        try:
            whole = int(v) if not isinstance(v, str) else None
        except (TypeError, ValueError, OverflowError):
            whole = None
        if whole is None or whole != v:
            raise MuonError(1, f"{what} must be an unsigned 64-bit integer")
        v = whole
    if not 0 <= v < 1 << 64:
        raise MuonError(1, f"{what} must be an unsigned 64-bit integer")
    return v


def layer_norm(x, gamma, beta, y, *, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """y = layer norm of x's rows (muon_layer_norm_fwd); gamma and beta may be
    None (1 and 0).  mean and rstd, float32 of one element a row, receive
    what layer_norm_backward needs."""
    rows, cols, ld = _matrix(x, "x")
    ld_y = _same(y, x, "y")
    wdt = _param_dtype(x, gamma, beta)
    g, b = _param(gamma, wdt, cols, "gamma"), _param(beta, wdt, cols, "beta")
    m, r = _flat(mean, rows, _F32, "mean"), _flat(rstd, rows, _F32, "rstd")
    dev, st = _device(stream, x, y, gamma, beta, mean, rstd)
    _call(dev, load_library().muon_layer_norm_fwd, x.data_ptr(), ld, _dtype_code(x.dtype), g, b,
          _dtype_code(wdt), rows, cols, eps, y.data_ptr(), ld_y, m, r, st)


@functools.lru_cache(maxsize=256)
def _norm_workspace(rows: int, cols: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_layer_norm_workspace_bytes(rows, cols, ctypes.byref(n)))
    return n.value


def layer_norm_backward(dy, x, gamma, mean, rstd, dx, *, dgamma=None, dbeta=None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of layer_norm (muon_layer_norm_bwd): dx, and dgamma and dbeta
    where given, in gamma's dtype (the `grads` of adamw_step)."""
    rows, cols, ld = _matrix(x, "x")
    ld_dy, ld_dx = _same(dy, x, "dy"), _same(dx, x, "dx")
    wdt = _param_dtype(x, gamma, dgamma, dbeta)
    g = _param(gamma, wdt, cols, "gamma")
    dg, db = _param(dgamma, wdt, cols, "dgamma"), _param(dbeta, wdt, cols, "dbeta")
    m, r = _flat(mean, rows, _F32, "mean"), _flat(rstd, rows, _F32, "rstd")
    dev, st = _device(stream, x, dy, dx, gamma, mean, rstd, dgamma, dbeta, workspace)
    keep, ws, ws_bytes = _workspace(workspace, _norm_workspace(rows, cols) if dg or db else 0, stream, dev, st)
    _call(dev, load_library().muon_layer_norm_bwd, dy.data_ptr(), ld_dy, x.data_ptr(), ld, _dtype_code(x.dtype), g,
          _dtype_code(wdt), m, r, rows, cols, dx.data_ptr(), ld_dx, dg, db, ws, ws_bytes, st)


def dropout(x, out, *, p: float, seed: int, offset: int = 0, offset_dev: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = [residual +] dropout(x) with a counter-based mask (muon_dropout).
    out may be x or residual itself.  The backward pass is the same call on
    the gradient, with the same p, seed and offset and no residual.
    offset_dev: an int64 tensor of one element added to offset on the device."""
    rows, cols, ld = _matrix(x, "x")
    ld_out = _same(out, x, "out")
    ld_res = 0 if residual is None else _same(residual, x, "residual")
    od = _flat(offset_dev, 1, _WORD, "offset_dev")
    dev, st = _device(stream, x, out, residual, offset_dev)
    _call(dev, load_library().muon_dropout, x.data_ptr(), ld, None if residual is None else residual.data_ptr(), ld_res,
          _dtype_code(x.dtype), rows, cols, p, _u64(seed, "seed"), _u64(offset, "offset"), od, out.data_ptr(), ld_out,
          st)


def dropout_add_layer_norm(x, residual, gamma, beta, h, y, *, p: float, seed: int, offset: int = 0,
                           offset_dev: Optional[torch.Tensor] = None, mean=None, rstd=None, eps: float = 1e-5,
                           stream=None) -> None:
    """h = residual + dropout(x) and y = layer norm of h in one pass
    (muon_dropout_add_layer_norm_fwd): the bits of dropout(residual=) followed
    by layer_norm.  h may be the residual itself."""
    rows, cols, ld = _matrix(x, "x")
    ld_res, ld_h, ld_y = _same(residual, x, "residual"), _same(h, x, "h"), _same(y, x, "y")
    wdt = _param_dtype(x, gamma, beta)
    g, b = _param(gamma, wdt, cols, "gamma"), _param(beta, wdt, cols, "beta")
    m, r = _flat(mean, rows, _F32, "mean"), _flat(rstd, rows, _F32, "rstd")
    od = _flat(offset_dev, 1, _WORD, "offset_dev")
    dev, st = _device(stream, x, residual, gamma, beta, h, y, mean, rstd, offset_dev)
    _call(dev, load_library().muon_dropout_add_layer_norm_fwd, x.data_ptr(), ld, residual.data_ptr(), ld_res,
          _dtype_code(x.dtype), g, b, _dtype_code(wdt), rows, cols, eps, p, _u64(seed, "seed"),
          _u64(offset, "offset"), od, h.data_ptr(), ld_h, y.data_ptr(), ld_y, m, r, st)


def dropout_add_layer_norm_backward(dy, h, gamma, mean, rstd, dx, dresidual, *, p: float, seed: int, offset: int = 0,
                                    offset_dev: Optional[torch.Tensor] = None, dh=None, dgamma=None, dbeta=None,
                                    workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of dropout_add_layer_norm (muon_dropout_add_layer_norm_bwd).
    dh is the gradient that reaches h by the residual path (None: 0);
    dresidual is the residual's gradient, dx that of x."""
    rows, cols, ld = _matrix(h, "h")
    ld_dy, ld_dx, ld_dres = _same(dy, h, "dy"), _same(dx, h, "dx"), _same(dresidual, h, "dresidual")
    ld_dh = 0 if dh is None else _same(dh, h, "dh")
    wdt = _param_dtype(h, gamma, dgamma, dbeta)
    g = _param(gamma, wdt, cols, "gamma")
    dg, db = _param(dgamma, wdt, cols, "dgamma"), _param(dbeta, wdt, cols, "dbeta")
    m, r = _flat(mean, rows, _F32, "mean"), _flat(rstd, rows, _F32, "rstd")
    od = _flat(offset_dev, 1, _WORD, "offset_dev")
    dev, st = _device(stream, h, dy, dx, dresidual, dh, gamma, mean, rstd, dgamma, dbeta, offset_dev, workspace)
    keep, ws, ws_bytes = _workspace(workspace, _norm_workspace(rows, cols) if dg or db else 0, stream, dev, st)
    _call(dev, load_library().muon_dropout_add_layer_norm_bwd, dy.data_ptr(), ld_dy,
          None if dh is None else dh.data_ptr(), ld_dh, h.data_ptr(), ld, _dtype_code(h.dtype), g, _dtype_code(wdt), m, r,
          rows, cols, p, _u64(seed, "seed"), _u64(offset, "offset"), od, dx.data_ptr(), ld_dx, dresidual.data_ptr(), ld_dres,
          dg, db, ws, ws_bytes, st)


def _choices(t: torch.Tensor, rows: int, dtypes, what: str, k: Optional[int] = None) -> int:
    """k of a [tokens, k] argument."""
    n = t.shape[-1] if t.dim() else 0
    if t.dim() < 1 or (k is not None and n != k):
        raise MuonError(2, f"{what} has shape {tuple(t.shape)}, expected [{rows}, {'k' if k is None else k}]")
    _flat(t, rows * n, dtypes, what)
    return n


@functools.lru_cache(maxsize=256)
def _route_workspace(rows: int, experts: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_route_workspace_bytes(rows, experts, ctypes.byref(n)))
    return n.value


def route(logits, indices, gates, counts, n_tokens, loss, *, coef: float = 1.0, renorm: bool = True, valid=None,
          prob_mean=None, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Top-k choices of every token's logits, their gates, the experts' counts
    and the balance loss (muon_route_fwd); k is indices.shape[-1].  valid: a
    uint8 or bool tensor, 0 for padding tokens."""
    rows, experts, ld = _matrix(logits, "logits")
    k = _choices(indices, rows, _I32, "indices")
    _choices(gates, rows, _F32, "gates", k)
    c, n = _flat(counts, experts, _I32, "counts"), _flat(n_tokens, 1, _I32, "n_tokens")
    lo, pm = _flat(loss, 1, _F32, "loss"), _flat(prob_mean, experts, _F32, "prob_mean")
    v = _flat(valid, rows, _MASK, "valid")
    dev, st = _device(stream, logits, indices, gates, counts, n_tokens, loss, valid, prob_mean, workspace)
    keep, ws, ws_bytes = _workspace(workspace, _route_workspace(rows, experts), stream, dev, st)
    _call(dev, load_library().muon_route_fwd, logits.data_ptr(), ld, _dtype_code(logits.dtype), rows, experts, k, v,
          1 if renorm else 0, coef, indices.data_ptr(), gates.data_ptr(), c, n, pm, lo, ws, ws_bytes, st)


def route_backward(logits, indices, counts, n_tokens, dlogits, *, dgates=None, dloss=None, coef: float = 1.0,
                   renorm: bool = True, valid=None, stream=None) -> None:
    """Gradient of route's gates and loss by the logits (muon_route_bwd).
    dgates (None: 0) and dloss (a device float; None: 1) are the gradients
    that reach them; coef, renorm and valid as in the forward call."""
    rows, experts, ld = _matrix(logits, "logits")
    ld_d = _same(dlogits, logits, "dlogits")
    k = _choices(indices, rows, _I32, "indices")
    if dgates is not None:
        _choices(dgates, rows, _F32, "dgates", k)
    c, n = _flat(counts, experts, _I32, "counts"), _flat(n_tokens, 1, _I32, "n_tokens")
    dl, v = _flat(dloss, 1, _F32, "dloss"), _flat(valid, rows, _MASK, "valid")
    dev, st = _device(stream, logits, indices, counts, n_tokens, dlogits, dgates, dloss, valid)
    _call(dev, load_library().muon_route_bwd, logits.data_ptr(), ld, _dtype_code(logits.dtype), rows, experts, k, v,
          1 if renorm else 0, coef, indices.data_ptr(), c, n, None if dgates is None else dgates.data_ptr(), dl,
          dlogits.data_ptr(), ld_d, st)
