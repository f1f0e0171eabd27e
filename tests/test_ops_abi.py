"""Refusals of the training operators that need no GPU: the C entry points
reject bad calls with the documented status before touching the device (fake
device pointers, never dereferenced), and the binding rejects tensors that
do not match."""
from __future__ import annotations

import ctypes

import pytest
import torch

from newton_schulz_05_amd import binding as B
from newton_schulz_05_amd import operators as O

F32, BF16 = B.MUON_F32, B.MUON_BF16
INVALID, SHAPE, DTYPE, WORKSPACE, ALIGN = 1, 2, 3, 5, 7
STEP = 1 << 24  # fake tensors lie this far apart
NAMES = ("x", "y", "gamma", "beta", "mean", "rstd", "dy", "dx", "dh", "dres", "dgamma", "dbeta", "res", "h", "ws", "od")
AT = {n: (i + 1) * STEP for i, n in enumerate(NAMES)}


def _detail():
    return B.load_library().muon_last_error_detail().decode()


def fwd(ld_x=64, dt=BF16, pdt=BF16, rows=4, cols=64, eps=1e-5, ld_y=64, **at):
    a = {**AT, **at}
    return B.load_library().muon_layer_norm_fwd(a["x"], ld_x, dt, a["gamma"], a["beta"], pdt, rows, cols, eps,
                                                a["y"], ld_y, a["mean"], a["rstd"], None)


def bwd(ld=64, dt=BF16, pdt=BF16, rows=400, cols=64, ws_bytes=1 << 20, **at):
    a = {**AT, **at}
    return B.load_library().muon_layer_norm_bwd(a["dy"], ld, a["x"], ld, dt, a["gamma"], pdt, a["mean"], a["rstd"],
                                                rows, cols, a["dx"], ld, a["dgamma"], a["dbeta"], a["ws"], ws_bytes,
                                                None)


def drop(ld=64, dt=BF16, rows=4, cols=64, p=0.1, ld_res=64, **at):
    a = {**AT, **at}
    return B.load_library().muon_dropout(a["x"], ld, a["res"], ld_res, dt, rows, cols, p, 1, 2, a["od"], a["y"], ld,
                                         None)


def fused(ld=64, dt=BF16, pdt=BF16, rows=4, cols=64, eps=1e-5, p=0.1, **at):
    a = {**AT, **at}
    return B.load_library().muon_dropout_add_layer_norm_fwd(
        a["x"], ld, a["res"], ld, dt, a["gamma"], a["beta"], pdt, rows, cols, eps, p, 1, 2, a["od"], a["h"], ld,
        a["y"], ld, a["mean"], a["rstd"], None)


def fused_bwd(ld=64, dt=BF16, pdt=BF16, rows=400, cols=64, p=0.1, ws_bytes=1 << 20, **at):
    a = {**AT, **at}
    return B.load_library().muon_dropout_add_layer_norm_bwd(
        a["dy"], ld, a["dh"], ld, a["h"], ld, dt, a["gamma"], pdt, a["mean"], a["rstd"], rows, cols, p, 1, 2, a["od"],
        a["dx"], ld, a["dres"], ld, a["dgamma"], a["dbeta"], a["ws"], ws_bytes, None)


RAT = {n: (i + 1) * STEP for i, n in enumerate(
    ("logits", "valid", "idx", "gates", "counts", "n", "mean", "loss", "ws", "dgates", "dloss", "dlogits"))}


def route(ld=8, dt=F32, tokens=1000, experts=8, k=2, renorm=1, coef=1.0, ws_bytes=1 << 20, **at):
    a = {**RAT, **at}
    return B.load_library().muon_route_fwd(a["logits"], ld, dt, tokens, experts, k, a["valid"], renorm, coef,
                                           a["idx"], a["gates"], a["counts"], a["n"], a["mean"], a["loss"], a["ws"],
                                           ws_bytes, None)


def route_bwd(ld=8, dt=F32, tokens=1000, experts=8, k=2, renorm=1, coef=1.0, ld_d=8, **at):
    a = {**RAT, **at}
    return B.load_library().muon_route_bwd(a["logits"], ld, dt, tokens, experts, k, a["valid"], renorm, coef,
                                           a["idx"], a["counts"], a["n"], a["dgates"], a["dloss"], a["dlogits"], ld_d,
                                           None)


@pytest.mark.parametrize("call", [fwd, bwd, fused, fused_bwd])
def test_norm_calls_reject_types_sizes_and_pointers(call):
    assert call(dt=7) == DTYPE
    assert call(pdt=-1) == DTYPE
    assert call(rows=-1) == SHAPE
    assert call(cols=0) == SHAPE
    assert call(cols=32769, **{"ld_x": 40000, "ld_y": 40000} if call is fwd else {"ld": 40000}) == SHAPE
    assert call(rows=(1 << 40) + 1) == SHAPE
    assert call(**{"ld_x" if call is fwd else "ld": 63}) == INVALID and "stride" in _detail()
    assert call(**{"ld_x" if call is fwd else "ld": 1 << 41}) == SHAPE
    big = ("h" if call is fused_bwd else "x")
    assert call(**{big: None}) == INVALID and "null" in _detail()
    assert call(**{big: AT[big] + 1}) == ALIGN
    assert call(gamma=AT["gamma"] + 1) == ALIGN
    assert call(mean=AT["mean"] + 2) == ALIGN


def test_forward_refusals():
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == INVALID
        assert fused(eps=eps) == INVALID
    assert fwd(y=AT["x"]) == INVALID and "overlap" in _detail()
    assert fwd(y=AT["x"] + 2 * 64 * 3) == INVALID
    assert fwd(mean=AT["x"] + 64) == INVALID
    assert fwd(rstd=AT["mean"] + 12) == INVALID
    assert fwd(y=AT["beta"]) == INVALID
    # interleaved column slices overlap once their columns do
    assert fwd(ld_x=128, ld_y=128, y=AT["x"] + 2 * 63) == INVALID
    assert fwd(ld_x=128, ld_y=128, y=AT["x"] + 2 * 65) == INVALID   # wraps into x's next row
    assert fwd(ld_x=128, ld_y=130, y=AT["x"] + 2 * 64) == INVALID   # strides differ: whole ranges
    assert fused(h=AT["x"]) == INVALID
    assert fused(y=AT["res"]) == INVALID
    assert fused(h=AT["res"] + 128) == INVALID
    assert fused(h=AT["y"]) == INVALID
    assert fused(y=AT["od"]) == INVALID
    # nothing to do: succeeds without touching a pointer
    none = dict.fromkeys(("x", "y", "gamma", "beta", "mean", "rstd", "res", "h", "od"))
    assert fwd(rows=0, **{n: none[n] for n in ("x", "y", "gamma", "beta", "mean", "rstd")}) == 0
    assert fused(rows=0, **none) == 0


def test_backward_refusals():
    for call in (bwd, fused_bwd):
        assert call(ws=None) == WORKSPACE
        assert call(ws=AT["ws"] + 8) == WORKSPACE
        n = ctypes.c_size_t()
        assert B.load_library().muon_layer_norm_workspace_bytes(400, 64, ctypes.byref(n)) == 0 and n.value > 0
        assert call(ws_bytes=n.value - 1) == WORKSPACE and str(n.value) in _detail()
        assert call(mean=None) == INVALID and call(rstd=None) == INVALID
        assert call(dx=AT["dy"]) == INVALID and "overlap" in _detail()
        assert call(dgamma=AT["dbeta"]) == INVALID
        assert call(dgamma=AT["gamma"]) == INVALID
        assert call(ws=AT["dx"]) == INVALID
        assert call(rows=0, dgamma=None, dbeta=None, ws=None) == 0
    assert fused_bwd(dres=AT["dx"]) == INVALID
    assert fused_bwd(dres=AT["dh"]) == INVALID
    assert fused_bwd(dres=None) == INVALID
    lib = B.load_library()
    assert lib.muon_layer_norm_workspace_bytes(4, 64, None) == INVALID
    assert lib.muon_layer_norm_workspace_bytes(4, 0, ctypes.byref(ctypes.c_size_t())) == SHAPE
    n = ctypes.c_size_t(1)
    assert lib.muon_layer_norm_workspace_bytes(1, 4096, ctypes.byref(n)) == 0 and n.value == 0


def test_dropout_refusals():
    for p in (-0.1, 1.1, float("nan")):
        assert drop(p=p) == INVALID
        assert fused(p=p) == INVALID
        assert fused_bwd(p=p) == INVALID
    assert drop(rows=1 << 32) == SHAPE
    assert drop(dt=9) == DTYPE
    assert drop(od=AT["od"] + 4) == ALIGN
    assert drop(cols=(1 << 34) + 1, ld=1 << 35, ld_res=1 << 35) == SHAPE
    assert drop(ld_res=63) == INVALID
    assert drop(x=None) == INVALID and drop(y=None) == INVALID
    assert drop(y=AT["x"] + 2) == INVALID       # shifted, not the same tensor
    assert drop(y=AT["res"] + 128) == INVALID
    assert drop(y=AT["res"], ld_res=65) == INVALID  # same address, other rows
    assert drop(y=AT["od"]) == INVALID
    assert drop(rows=0, x=None, y=None, res=None) == 0


def test_route_refusals():
    for call in (route, route_bwd):
        assert call(dt=3) == DTYPE
        assert call(experts=0) == SHAPE
        assert call(experts=1025, ld=1025, **({"ld_d": 1025} if call is route_bwd else {})) == SHAPE
        assert call(k=0) == SHAPE and call(k=9) == SHAPE
        assert call(experts=64, ld=64, k=17, **({"ld_d": 64} if call is route_bwd else {})) == SHAPE
        assert call(tokens=-1) == SHAPE
        assert call(tokens=1 << 30) == SHAPE   # tokens * k needs more than 31 bits
        assert call(ld=7) == INVALID
        assert call(renorm=2) == INVALID
        assert call(coef=float("nan")) == INVALID
        assert call(logits=None) == INVALID
        assert call(logits=RAT["logits"] + 2) == ALIGN
        assert call(idx=RAT["idx"] + 1) == ALIGN
        assert call(counts=None) == INVALID and call(n=None) == INVALID and call(idx=None) == INVALID
    assert route(loss=None) == INVALID and route(gates=None) == INVALID
    assert route(ws=None) == WORKSPACE and route(ws=RAT["ws"] + 4) == WORKSPACE and route(ws_bytes=64) == WORKSPACE
    assert route(gates=RAT["idx"] + 4) == INVALID
    assert route(counts=RAT["n"]) == INVALID
    assert route(mean=RAT["logits"] + 64) == INVALID
    assert route(ws=RAT["valid"]) == INVALID
    assert route_bwd(dlogits=RAT["logits"]) == INVALID
    assert route_bwd(ld_d=7) == INVALID
    assert route_bwd(dlogits=None) == INVALID
    assert route_bwd(tokens=0, logits=None, dlogits=None, idx=None, dgates=None, valid=None) == 0
    lib = B.load_library()
    assert lib.muon_route_workspace_bytes(100, 8, None) == INVALID
    n = ctypes.c_size_t()
    assert lib.muon_route_workspace_bytes(100, 1025, ctypes.byref(n)) == SHAPE
    assert lib.muon_route_workspace_bytes(0, 8, ctypes.byref(n)) == 0 and n.value == 0


# ---- the binding -------------------------------------------------------------------

def _status(f, *a, **k):
    with pytest.raises(B.MuonError) as e:
        f(*a, **k)
    return e.value.status


def test_binding_rejects_host_tensors_and_mismatches():
    x, y = torch.zeros(4, 8), torch.zeros(4, 8)
    g = torch.zeros(8)
    f1 = torch.zeros(4)
    assert _status(O.layer_norm, x, g, None, y) == INVALID            # host tensors
    assert _status(O.layer_norm, x, g, None, y.bfloat16()) == DTYPE
    assert _status(O.layer_norm, x, g, None, torch.zeros(4, 9)) == SHAPE
    assert _status(O.layer_norm, x, torch.zeros(9), None, y) == SHAPE
    assert _status(O.layer_norm, x, g, g.bfloat16(), y) == DTYPE
    assert _status(O.layer_norm, x, g, g, y, mean=torch.zeros(5)) == SHAPE
    assert _status(O.layer_norm, x, g, g, y, mean=f1.double()) == DTYPE
    assert _status(O.layer_norm, x.t(), g, None, y.t()) == INVALID    # columns, not rows
    assert _status(O.layer_norm, torch.zeros(()), g, None, y) == SHAPE
    assert _status(O.layer_norm, torch.zeros(4, 6, 8)[:, :3], g, None, torch.zeros(4, 3, 8)) == INVALID
    # a broadcast gradient has no rows of its own
    assert _status(O.layer_norm_backward, torch.zeros(1, 1).expand(4, 8), x, g, f1, f1, y) == INVALID
    assert _status(O.layer_norm_backward, y, x, g, f1, f1, torch.zeros(4, 8), dgamma=g.bfloat16()) == DTYPE
    assert _status(O.dropout, x, y, p=0.1, seed=-1) == INVALID
    assert _status(O.dropout, x, y, p=0.1, seed=0, offset_dev=torch.zeros(1)) == DTYPE
    assert _status(O.dropout, x, y, p=0.1, seed=0, residual=torch.zeros(4, 8).half()) == DTYPE
    i, c = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    one, w = torch.zeros(1), torch.zeros(4, 2)
    n = torch.zeros(1, dtype=torch.int32)
    assert _status(O.route, x, i.long(), w, c, n, one) == DTYPE
    assert _status(O.route, x, i, torch.zeros(4, 3), c, n, one) == SHAPE
    assert _status(O.route, x, i, w, c[:7], n, one) == SHAPE
    assert _status(O.route, x, i, w, c, n, one, valid=torch.ones(4)) == DTYPE
    assert _status(O.route, x, i, w, c, n, one) == INVALID
    assert _status(O.route_backward, x, i, c, n, torch.zeros(4, 9)) == SHAPE


def test_matrix_arguments():
    assert O._matrix(torch.zeros(3, 4, 8), "x") == (12, 8, 8)
    assert O._matrix(torch.zeros(3, 4, 20)[:, :, 2:10], "x") == (12, 8, 20)
    assert O._matrix(torch.zeros(8), "x") == (1, 8, 8)
    assert O._matrix(torch.zeros(1, 8), "x") == (1, 8, 8)
    assert O._matrix(torch.zeros(5, 1, 8), "x") == (5, 8, 8)
    assert O._matrix(torch.zeros(0, 8), "x")[0] == 0
    assert O._matrix(torch.zeros(3, 0, 8), "x")[0] == 0
    assert O._matrix(torch.zeros(6, 9)[::2], "x") == (3, 9, 18)
    assert O._matrix(torch.zeros(9, 1).t(), "x") == (1, 9, 9)
