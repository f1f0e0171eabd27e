"""Binding of the training operators beside the step (include/muon.h): layer
norm, dropout, the two fused with the residual add, the expert router, the norm
and rotation of query and key heads, token log-probabilities, and the policy and
preference losses on them.

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

from .binding import MUON_BF16, MUON_F32, MuonError, MuonHeadStrides, _check, load_library


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


@functools.lru_cache(maxsize=1024)
def _head_strides(stride: Tuple[int, ...], dim: int):
    """(structure, its address) of a muon_head_strides for a tensor's strides;
    None where the last dimension is not contiguous."""
    if stride[-1] != 1 and dim > 1:
        return None
    s = MuonHeadStrides(stride[0] if len(stride) == 4 else 0, stride[-3], stride[-2])
    return s, ctypes.addressof(s)


# The operators from here on check an argument's device with the argument itself,
# against that of the call's first tensor, and that one at the end (_stream): one
# look at each tensor instead of two.

def _elsewhere(t: torch.Tensor, what: str, dev: int) -> MuonError:
    return MuonError(1, f"{what} is on device {t.get_device()}, expected {dev}" if t.get_device() >= 0
                     else "every tensor must be a device tensor")


def _heads(t: torch.Tensor, shape, dt: torch.dtype, what: str, dev: int):
    """Strides' structure of a tensor of heads of this shape, dtype and device."""
    if t.shape != shape:
        raise MuonError(2, f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dt:
        raise MuonError(3, f"{what} has dtype {t.dtype}, expected {dt}")
    s = _head_strides(t.stride(), shape[-1])
    if s is None:
        raise MuonError(1, f"{what}: the last dimension is not contiguous")
    if t.get_device() != dev:
        raise _elsewhere(t, what, dev)
    return s


def _gain(t: Optional[torch.Tensor], dt: torch.dtype, n: int, what: str, dev: int) -> Optional[int]:
    """_param, with the device."""
    if t is None:
        return None
    if t.dtype is dt and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _param(t, dt, n, what)
    raise _elsewhere(t, what, dev)


def _vec(t: Optional[torch.Tensor], n: int, what: str, dev: int) -> Optional[int]:
    """_flat of a float32 argument, with the device."""
    if t is None:
        return None
    if t.dtype is torch.float32 and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _flat(t, n, _F32, what)
    raise _elsewhere(t, what, dev)


def _words(t: Optional[torch.Tensor], n: int, what: str, dev: int) -> Optional[int]:
    """_flat of an int64 argument, with the device."""
    if t is None:
        return None
    if t.dtype is torch.int64 and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _flat(t, n, _WORD, what)
    raise _elsewhere(t, what, dev)


def _stream(stream, dev: int) -> int:
    """Stream handle of a call on device `dev` (see _device)."""
    if dev < 0:
        raise MuonError(1, "every tensor must be a device tensor")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise MuonError(1, f"a stream of {stream.device} for tensors on device {dev}")
    return stream.cuda_stream


def _scratch(given: Optional[torch.Tensor], need: int, stream, dev: int, handle: int):
    """_workspace, with the device."""
    if given is None and need == 0:
        return None, None, 0
    if given is not None and given.get_device() != dev:
        raise _elsewhere(given, "workspace", dev)
    return _workspace(given, need, stream, dev, handle)


def _head_sizes(shape, keys) -> Tuple[int, int, int, int, int]:
    """(batch, tokens, query heads, key heads, dim) of the shapes of q and k."""
    if len(shape) == 4:
        batch, tokens, hq, dim = shape
    elif len(shape) == 3:
        tokens, hq, dim = shape
        batch = 1
    else:
        raise MuonError(2, f"q has {len(shape)} dimensions, expected [batch, tokens, heads, dim] or [tokens, heads, dim]")
    if keys is None:
        return batch, tokens, hq, 0, dim
    if len(keys) != len(shape) or keys[-1] != dim or keys[-3] != tokens or (len(keys) == 4 and keys[0] != batch):
        raise MuonError(2, f"k has shape {tuple(keys)}, q {tuple(shape)}: they may differ in their heads only")
    return batch, tokens, hq, keys[-2], dim


def _angles(cos, sin, positions, batch: int, tokens: int, dev: int) -> Tuple:
    """(cos, sin, table rows, rot, positions, their batch stride)."""
    if cos is None or sin is None:
        if cos is not sin:
            raise MuonError(1, "cos and sin come together")
        return None, None, 0, 0, None, 0
    shape = cos.shape
    if len(shape) != 2 or sin.shape != shape:
        raise MuonError(2, f"cos and sin have shapes {tuple(shape)} and {tuple(sin.shape)}, expected [table rows, rot / 2]")
    rows, half = shape
    c, s = _vec(cos, rows * half, "cos", dev), _vec(sin, rows * half, "sin", dev)
    if positions is None:
        return c, s, rows, 2 * half, None, 0
    if positions.dtype is not torch.int64:
        raise MuonError(3, f"positions has dtype {positions.dtype}, expected torch.int64")
    shape, stride = positions.shape, positions.stride()
    each = 0
    if shape == (batch, tokens):
        if batch > 1:
            each = stride[0]
            if each != 0 and each < tokens:
                raise MuonError(1, "positions: the sequences overlap")
    elif shape != (tokens,):
        raise MuonError(2, f"positions has shape {tuple(shape)}, expected ({tokens},) or ({batch}, {tokens})")
    if tokens > 1 and stride[-1] != 1:
        raise MuonError(1, "positions: the last dimension is not contiguous")
    if positions.get_device() != dev:
        raise _elsewhere(positions, "positions", dev)
    return c, s, rows, 2 * half, positions.data_ptr(), each


_NO_STRIDES = (None, None)


def qk_norm_rope(q, k, gamma_q, gamma_k, cos, sin, q_out, k_out, *, positions=None, interleaved: bool = False,
                 eps: float = 1e-6, stream=None) -> None:
    """q_out and k_out = the heads of q and k divided by their root mean square,
    times gamma, their first 2 * cos.shape[1] elements turned by the tokens'
    angles (muon_qk_norm_rope_fwd).  Heads are tensors [batch, tokens, heads,
    dim] or [tokens, heads, dim] of any order in memory (slices of a projection's
    output, transposed ones); k, gamma_k and k_out may be None.  cos and sin:
    [table rows, rot / 2] float32, or None for no rotation.  positions: int64,
    [batch, tokens] or [tokens] (None: 0, 1, ...): the rows of cos and sin; a
    token whose position has no row is not turned.  q_out may be q itself, k_out k
    itself."""
    shape, dt, keys = q.shape, q.dtype, None if k is None else k.shape
    batch, tokens, hq, hk, dim = _head_sizes(shape, keys)
    dev = q.get_device()
    sq, sqo = _heads(q, shape, dt, "q", dev), _heads(q_out, shape, dt, "q_out", dev)
    if k is None:
        if k_out is not None:
            raise MuonError(1, "k and k_out come together")
        kp = kop = None
        sk = sko = _NO_STRIDES
    else:
        if k_out is None:
            raise MuonError(1, "k and k_out come together")
        sk, sko = _heads(k, keys, dt, "k", dev), _heads(k_out, keys, dt, "k_out", dev)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    wdt = _param_dtype(q, gamma_q, gamma_k)
    gq, gk = _gain(gamma_q, wdt, dim, "gamma_q", dev), _gain(gamma_k, wdt, dim, "gamma_k", dev)
    c, s, rows, rot, pos, each = _angles(cos, sin, positions, batch, tokens, dev)
    st = _stream(stream, dev)
    _call(dev, load_library().muon_qk_norm_rope_fwd, q.data_ptr(), sq[1], kp, sk[1], _dtype_code(dt), batch, tokens, hq, hk,
          dim, gq, gk, _dtype_code(wdt), eps, c, s, rows, rot, 1 if interleaved else 0, pos, each, q_out.data_ptr(), sqo[1],
          kop, sko[1], st)


@functools.lru_cache(maxsize=256)
def _heads_workspace(rows_q: int, rows_k: int, dim: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_qk_norm_rope_workspace_bytes(rows_q, rows_k, dim, ctypes.byref(n)))
    return n.value


def qk_norm_rope_backward(dq_out, dk_out, q, k, gamma_q, gamma_k, cos, sin, dq, dk, *, dgamma_q=None, dgamma_k=None,
                          positions=None, interleaved: bool = False, eps: float = 1e-6,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of qk_norm_rope (muon_qk_norm_rope_bwd) from those that reach
    q_out and k_out and the forward call's q and k: dq and dk, and dgamma_q and
    dgamma_k where given, in the gains' dtype (the `grads` of adamw_step).  dq
    may be dq_out itself, dk dk_out itself."""
    shape, dt, keys = q.shape, q.dtype, None if k is None else k.shape
    batch, tokens, hq, hk, dim = _head_sizes(shape, keys)
    dev = q.get_device()
    sq, sdqo, sdq = _heads(q, shape, dt, "q", dev), _heads(dq_out, shape, dt, "dq_out", dev), _heads(dq, shape, dt, "dq", dev)
    if k is None:
        if dk_out is not None or dk is not None:
            raise MuonError(1, "k, dk_out and dk come together")
        kp = dkop = dkp = None
        sk = sdko = sdk = _NO_STRIDES
    else:
        if dk_out is None or dk is None:
            raise MuonError(1, "k, dk_out and dk come together")
        sk, sdko, sdk = _heads(k, keys, dt, "k", dev), _heads(dk_out, keys, dt, "dk_out", dev), _heads(dk, keys, dt, "dk", dev)
        kp, dkop, dkp = k.data_ptr(), dk_out.data_ptr(), dk.data_ptr()
    wdt = _param_dtype(q, gamma_q, gamma_k, dgamma_q, dgamma_k)
    gq, gk = _gain(gamma_q, wdt, dim, "gamma_q", dev), _gain(gamma_k, wdt, dim, "gamma_k", dev)
    dgq, dgk = _gain(dgamma_q, wdt, dim, "dgamma_q", dev), _gain(dgamma_k, wdt, dim, "dgamma_k", dev)
    c, s, rows, rot, pos, each = _angles(cos, sin, positions, batch, tokens, dev)
    st = _stream(stream, dev)
    need = _heads_workspace(batch * tokens * hq, batch * tokens * hk, dim) if dgq or dgk else 0
    keep, ws, ws_bytes = _scratch(workspace, need, stream, dev, st)
    _call(dev, load_library().muon_qk_norm_rope_bwd, dq_out.data_ptr(), sdqo[1], dkop, sdko[1], q.data_ptr(), sq[1], kp,
          sk[1], _dtype_code(dt), batch, tokens, hq, hk, dim, gq, gk, _dtype_code(wdt), eps, c, s, rows, rot,
          1 if interleaved else 0, pos, each, dq.data_ptr(), sdq[1], dkp, sdk[1], dgq, dgk, ws, ws_bytes, st)


@functools.lru_cache(maxsize=256)
def _logp_workspace(rows: int, vocab: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_token_logp_workspace_bytes(rows, vocab, ctypes.byref(n)))
    return n.value


def token_logp(logits, targets, logp, lse, *, scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """logp = log softmax(scale * logits) of every token's target, lse = log of
    the softmax's sum (muon_token_logp_fwd).  targets: int64, one a token; one
    outside the vocabulary (a prompt or padding token) gives 0 in both."""
    rows, vocab, ld = _matrix(logits, "logits")
    dev = logits.get_device()
    t = _words(targets, rows, "targets", dev)
    lp, ls = _vec(logp, rows, "logp", dev), _vec(lse, rows, "lse", dev)
    st = _stream(stream, dev)
    keep, ws, ws_bytes = _scratch(workspace, _logp_workspace(rows, vocab), stream, dev, st)
    _call(dev, load_library().muon_token_logp_fwd, logits.data_ptr(), ld, _dtype_code(logits.dtype), rows, vocab, t,
          scale, lp, ls, ws, ws_bytes, st)


def token_logp_backward(logits, targets, logp, lse, dlogp, dlogits, *, scale: float = 1.0, stream=None) -> None:
    """Gradient of token_logp's logp by the logits (muon_token_logp_bwd), from
    the logp and lse that it wrote and the gradient dlogp that reaches logp.
    dlogits may be logits itself."""
    rows, vocab, ld = _matrix(logits, "logits")
    dev = logits.get_device()
    ld_d = _same(dlogits, logits, "dlogits")
    if dlogits.get_device() != dev:
        raise _elsewhere(dlogits, "dlogits", dev)
    t = _words(targets, rows, "targets", dev)
    lp, ls, d = _vec(logp, rows, "logp", dev), _vec(lse, rows, "lse", dev), _vec(dlogp, rows, "dlogp", dev)
    st = _stream(stream, dev)
    _call(dev, load_library().muon_token_logp_bwd, logits.data_ptr(), ld, _dtype_code(logits.dtype), rows, vocab, t,
          scale, lp, ls, d, dlogits.data_ptr(), ld_d, st)


@functools.lru_cache(maxsize=256)
def _policy_workspace(tokens: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_policy_loss_workspace_bytes(tokens, ctypes.byref(n)))
    return n.value


def policy_loss(logp, old_logp, advantages, loss, *, ref_logp=None, weight=None, dlogp=None, dloss=None, terms=None,
                clip_low: float = 0.2, clip_high: float = 0.2, beta: float = 0.0,
                workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Clipped policy loss with a KL term, and its gradient dlogp where given
    (muon_policy_loss): the loss is the sum of weight times a token's term, so
    weight is 1 / n for a mean and 0 for tokens that do not count.  old_logp
    None: logp itself (ratio 1); ref_logp None: no KL term; dloss, a device
    float: what dlogp is multiplied by.  terms receives the policy sum, the KL sum
    and the weight of the clipped tokens."""
    n, dev = logp.numel(), logp.get_device()
    lp, ol = _vec(logp, n, "logp", dev), _vec(old_logp, n, "old_logp", dev)
    rf, ad = _vec(ref_logp, n, "ref_logp", dev), _vec(advantages, n, "advantages", dev)
    w, g = _vec(weight, n, "weight", dev), _vec(dlogp, n, "dlogp", dev)
    up, lo, tm = _vec(dloss, 1, "dloss", dev), _vec(loss, 1, "loss", dev), _vec(terms, 3, "terms", dev)
    st = _stream(stream, dev)
    keep, ws, ws_bytes = _scratch(workspace, _policy_workspace(n), stream, dev, st)
    _call(dev, load_library().muon_policy_loss, lp, ol, rf, ad, w, n, clip_low, clip_high, beta, up, lo, tm, g, ws,
          ws_bytes, st)


@functools.lru_cache(maxsize=256)
def _preference_workspace(tokens: int, pairs: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().muon_preference_loss_workspace_bytes(tokens, pairs, ctypes.byref(n)))
    return n.value


def preference_loss(logp, offsets, loss, *, ref_logp=None, valid=None, weight=None, rewards=None, dlogp=None, dloss=None,
                    beta: float = 0.1, margin: float = 0.0, smoothing: float = 0.0, average: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Preference loss on pairs of answers, and its gradient dlogp where given
    (muon_preference_loss).  offsets: int64, 2 * pairs + 1 rising ends of the
    answers in logp, the preferred ones of all pairs first.  valid: uint8 or bool,
    0 for tokens that do not count; weight: one a pair (None: 1 / pairs);
    rewards receives beta times each answer's log-ratio (average: its mean)."""
    n, ends, dev = logp.numel(), offsets.numel(), logp.get_device()
    if ends % 2 == 0:
        raise MuonError(2, f"offsets has {ends} elements, expected 2 * pairs + 1")
    pairs = ends // 2
    lp, rf = _vec(logp, n, "logp", dev), _vec(ref_logp, n, "ref_logp", dev)
    v, off = _flat(valid, n, _MASK, "valid"), _words(offsets, ends, "offsets", dev)
    if valid is not None and valid.get_device() != dev:
        raise _elsewhere(valid, "valid", dev)
    w, rw = _vec(weight, pairs, "weight", dev), _vec(rewards, 2 * pairs, "rewards", dev)
    g, up, lo = _vec(dlogp, n, "dlogp", dev), _vec(dloss, 1, "dloss", dev), _vec(loss, 1, "loss", dev)
    st = _stream(stream, dev)
    keep, ws, ws_bytes = _scratch(workspace, _preference_workspace(n, pairs), stream, dev, st)
    _call(dev, load_library().muon_preference_loss, lp, rf, v, n, off, pairs, w, beta, margin, smoothing,
          1 if average else 0, up, lo, rw, g, ws, ws_bytes, st)
