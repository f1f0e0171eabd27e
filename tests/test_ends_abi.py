"""Refusals of the operators at the two ends of a training step that need no
GPU: the C entry points reject bad calls with the documented status before
touching the device (fake device pointers, never dereferenced), and the binding
rejects tensors that do not match."""
from __future__ import annotations

import ctypes

import pytest
import torch

from newton_schulz_05_amd import binding as B
from newton_schulz_05_amd import operators as O

F32, BF16 = B.MUON_F32, B.MUON_BF16
INVALID, SHAPE, DTYPE, WORKSPACE, ALIGN = 1, 2, 3, 5, 7
STEP = 1 << 26  # fake tensors lie this far apart
INF, NAN = float("inf"), float("nan")


def _detail():
    return B.load_library().muon_last_error_detail().decode()


def _at(*names):
    return {n: (i + 1) * STEP for i, n in enumerate(names)}


# ---- heads: 2 x 5 tokens, 4 and 2 heads of 16, contiguous unless told otherwise
HAT = _at("q", "k", "qo", "ko", "dqo", "dko", "dq", "dk", "gq", "gk", "dgq", "dgk", "cos", "sin", "pos", "ws")
PLAIN_Q, PLAIN_K = (5 * 64, 64, 16), (5 * 32, 32, 16)


def _strides(s):
    return None if s is None else ctypes.addressof(_keep.setdefault(s, B.MuonHeadStrides(*s)))


_keep = {}


def fwd(dt=BF16, pdt=BF16, batch=2, tokens=5, hq=4, hk=2, dim=16, eps=1e-6, table=9, rot=16, inter=0, posb=5,
        sq=PLAIN_Q, sk=PLAIN_K, sqo=PLAIN_Q, sko=PLAIN_K, **at):
    a = {**HAT, **at}
    return B.load_library().muon_qk_norm_rope_fwd(
        a["q"], _strides(sq), a["k"], _strides(sk), dt, batch, tokens, hq, hk, dim, a["gq"], a["gk"], pdt, eps, a["cos"],
        a["sin"], table, rot, inter, a["pos"], posb, a["qo"], _strides(sqo), a["ko"], _strides(sko), None)


def bwd(dt=BF16, pdt=BF16, batch=2, tokens=5, hq=4, hk=2, dim=16, eps=1e-6, table=9, rot=16, inter=0, posb=5,
        sq=PLAIN_Q, sk=PLAIN_K, sdqo=PLAIN_Q, sdko=PLAIN_K, sdq=PLAIN_Q, sdk=PLAIN_K, ws_bytes=1 << 20, **at):
    a = {**HAT, **at}
    return B.load_library().muon_qk_norm_rope_bwd(
        a["dqo"], _strides(sdqo), a["dko"], _strides(sdko), a["q"], _strides(sq), a["k"], _strides(sk), dt, batch, tokens,
        hq, hk, dim, a["gq"], a["gk"], pdt, eps, a["cos"], a["sin"], table, rot, inter, a["pos"], posb, a["dq"],
        _strides(sdq), a["dk"], _strides(sdk), a["dgq"], a["dgk"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_heads_reject_types_sizes_and_pointers(call):
    assert call(dt=7) == DTYPE and call(pdt=-1) == DTYPE
    assert call(batch=-1) == SHAPE and call(tokens=-1) == SHAPE
    assert call(dim=0) == SHAPE and call(dim=513) == SHAPE
    assert call(hq=0) == SHAPE and call(hk=0) == SHAPE and call(hk=-1) == SHAPE
    assert call(batch=1 << 20, tokens=1 << 20) == SHAPE
    assert call(batch=1 << 31, tokens=1 << 62) == SHAPE
    for eps in (0.0, -1e-6, NAN, INF):
        assert call(eps=eps) == INVALID
    assert call(inter=2) == INVALID
    assert call(rot=15) == SHAPE and call(rot=18) == SHAPE and call(rot=-2) == SHAPE
    assert call(table=-1) == SHAPE and call(table=1 << 50) == SHAPE
    assert call(cos=None) == INVALID and call(sin=None) == INVALID
    assert call(posb=4) == INVALID and call(posb=-1) in (INVALID, SHAPE) and call(posb=1 << 50) == SHAPE
    assert call(q=None) == INVALID and "null" in _detail()
    assert call(k=None) == INVALID
    assert call(q=HAT["q"] + 1) == ALIGN and call(cos=HAT["cos"] + 2) == ALIGN and call(pos=HAT["pos"] + 4) == ALIGN
    assert call(gq=HAT["gq"] + 1) == ALIGN
    assert call(sq=None) == INVALID and "strides" in _detail()
    assert call(sq=(5 * 64, 64, 15)) == INVALID and "nest" in _detail()
    assert call(sq=(64, 5 * 64, -16)) == INVALID
    assert call(sq=(0, 64, 16)) == INVALID          # a broadcast batch
    assert call(sq=(5 * 64, 48, 16)) == INVALID     # tokens overlap
    assert call(sq=(1 << 41, 64, 16)) == SHAPE


def test_heads_forward_refusals():
    assert fwd(qo=None) == INVALID and fwd(ko=None) == INVALID
    assert fwd(qo=HAT["q"] + 64) == INVALID and "overlap" in _detail()
    assert fwd(qo=HAT["q"], sqo=(64, 128, 16)) == INVALID       # the same tensor in another order
    assert fwd(ko=HAT["q"]) == INVALID
    assert fwd(qo=HAT["ko"]) == INVALID
    assert fwd(qo=HAT["cos"]) == INVALID and fwd(ko=HAT["pos"]) == INVALID and fwd(qo=HAT["gk"]) == INVALID
    # slices of one buffer of 8 heads: apart as long as their heads are
    packed = (5 * 128, 128, 16)
    assert fwd(sqo=packed, sko=packed, ko=HAT["qo"] + 2 * 48) == INVALID
    # nothing to do: succeeds without touching a pointer
    none = dict.fromkeys(HAT)
    assert fwd(batch=0, table=0, **none) == 0 and fwd(tokens=0, rot=0, **none) == 0
    alone = dict(k=None, ko=None, gk=None, sk=None, sko=None)
    assert fwd(hk=1, **alone) == INVALID
    assert fwd(tokens=0, hk=0, **alone) == 0


def test_heads_backward_refusals():
    lib = B.load_library()
    big = dict(tokens=500, posb=500, sq=(32000, 64, 16), sk=(16000, 32, 16), sdqo=(32000, 64, 16), sdko=(16000, 32, 16),
               sdq=(32000, 64, 16), sdk=(16000, 32, 16))
    n = ctypes.c_size_t()
    assert lib.muon_qk_norm_rope_workspace_bytes(4000, 2000, 16, ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(ws=None, **big) == WORKSPACE and bwd(ws=HAT["ws"] + 8, **big) == WORKSPACE
    assert bwd(ws_bytes=n.value - 1, **big) == WORKSPACE and str(n.value) in _detail()
    assert bwd(dqo=None) == INVALID and bwd(dq=None) == INVALID and bwd(dko=None) == INVALID and bwd(dk=None) == INVALID
    assert bwd(dq=HAT["q"]) == INVALID and "overlap" in _detail()   # only the gradient may be the output
    assert bwd(dq=HAT["dqo"], sdq=(64, 128, 16)) == INVALID
    assert bwd(dk=HAT["dqo"]) == INVALID
    assert bwd(dgq=HAT["dgk"]) == INVALID and bwd(dgq=HAT["gq"]) == INVALID and bwd(dgk=HAT["dk"]) == INVALID
    assert bwd(ws=HAT["dq"], **big) == INVALID
    assert bwd(dgq=HAT["dgq"] + 1) == ALIGN
    none = dict.fromkeys(HAT)
    assert bwd(batch=0, table=0, **none) == 0
    alone = dict(k=None, dko=None, dk=None, gk=None, sk=None, sdko=None, sdk=None, hk=0)
    assert bwd(**alone) == INVALID and "dgamma_k" in _detail()
    assert lib.muon_qk_norm_rope_workspace_bytes(10, 10, 16, None) == INVALID
    assert lib.muon_qk_norm_rope_workspace_bytes(10, -1, 16, ctypes.byref(n)) == SHAPE
    assert lib.muon_qk_norm_rope_workspace_bytes(10, 10, 513, ctypes.byref(n)) == SHAPE
    assert lib.muon_qk_norm_rope_workspace_bytes(1, 0, 16, ctypes.byref(n)) == 0 and n.value == 0


# ---- token log-probabilities
LAT = _at("x", "t", "lp", "lse", "d", "dx", "ws")


def logp(ld=80000, dt=BF16, tokens=3, vocab=80000, scale=1.0, ws_bytes=1 << 20, **at):
    a = {**LAT, **at}
    return B.load_library().muon_token_logp_fwd(a["x"], ld, dt, tokens, vocab, a["t"], scale, a["lp"], a["lse"], a["ws"],
                                                ws_bytes, None)


def logp_bwd(ld=80000, dt=BF16, tokens=3, vocab=80000, scale=1.0, ld_d=80000, **at):
    a = {**LAT, **at}
    return B.load_library().muon_token_logp_bwd(a["x"], ld, dt, tokens, vocab, a["t"], scale, a["lp"], a["lse"], a["d"],
                                                a["dx"], ld_d, None)


def test_token_logp_refusals():
    for call in (logp, logp_bwd):
        assert call(dt=5) == DTYPE
        assert call(tokens=-1) == SHAPE and call(tokens=1 << 31) == SHAPE and call(vocab=0) == SHAPE
        wide = dict(ld=1 << 25, vocab=(1 << 24) + 1, **(dict(ld_d=1 << 25) if call is logp_bwd else {}))
        assert call(**wide) == SHAPE
        assert call(ld=79999) == INVALID
        for s in (0.0, -1.0, NAN, INF, 1e31):
            assert call(scale=s) == INVALID
        for n in ("x", "t", "lp", "lse"):
            assert call(**{n: None}) == INVALID
        assert call(x=LAT["x"] + 1) == ALIGN and call(t=LAT["t"] + 4) == ALIGN and call(lp=LAT["lp"] + 2) == ALIGN
    assert logp(lse=LAT["lp"] + 8) == INVALID and logp(lp=LAT["x"] + 64) == INVALID and logp(lse=LAT["t"]) == INVALID
    assert logp(ws=None) == WORKSPACE and logp(ws_bytes=16) == WORKSPACE and logp(ws=LAT["ws"] + 4) == WORKSPACE
    assert logp(ws=LAT["x"]) == INVALID
    assert logp(tokens=0, x=None, t=None, lp=None, lse=None, ws=None) == 0
    assert logp_bwd(dx=LAT["x"] + 2) == INVALID       # shifted, not the logits themselves
    assert logp_bwd(dx=LAT["x"], ld_d=80001) == INVALID
    assert logp_bwd(dx=LAT["d"]) == INVALID and logp_bwd(d=None) == INVALID and logp_bwd(dx=None) == INVALID
    assert logp_bwd(ld_d=7) == INVALID
    assert logp_bwd(tokens=0, x=None, t=None, lp=None, lse=None, d=None, dx=None) == 0
    lib, n = B.load_library(), ctypes.c_size_t(1)
    assert lib.muon_token_logp_workspace_bytes(1, 100, None) == INVALID
    assert lib.muon_token_logp_workspace_bytes(1, 0, ctypes.byref(n)) == SHAPE
    assert lib.muon_token_logp_workspace_bytes(1, 100, ctypes.byref(n)) == 0 and n.value == 0


# ---- losses
PAT = _at("lp", "old", "ref", "adv", "w", "up", "loss", "terms", "d", "ws", "valid", "off", "rew")


def policy(tokens=5000, low=0.2, high=0.2, beta=0.1, ws_bytes=1 << 20, **at):
    a = {**PAT, **at}
    return B.load_library().muon_policy_loss(a["lp"], a["old"], a["ref"], a["adv"], a["w"], tokens, low, high, beta,
                                             a["up"], a["loss"], a["terms"], a["d"], a["ws"], ws_bytes, None)


def pref(tokens=500, pairs=30, beta=0.1, margin=0.0, smoothing=0.1, average=0, ws_bytes=1 << 20, **at):
    a = {**PAT, **at}
    return B.load_library().muon_preference_loss(a["lp"], a["ref"], a["valid"], tokens, a["off"], pairs, a["w"], beta, margin,
                                                 smoothing, average, a["up"], a["loss"], a["rew"], a["d"], a["ws"], ws_bytes,
                                                 None)


def test_policy_refusals():
    assert policy(tokens=-1) == SHAPE and policy(tokens=(1 << 40) + 1) == SHAPE
    for v in (-0.1, 1.1, NAN):
        assert policy(low=v) == INVALID
    for v in (-0.1, INF, NAN):
        assert policy(high=v) == INVALID
    assert policy(beta=NAN) == INVALID and policy(beta=INF) == INVALID
    for n in ("lp", "adv", "loss"):
        assert policy(**{n: None}) == INVALID
    assert policy(d=PAT["lp"]) == INVALID and "overlap" in _detail()
    assert policy(loss=PAT["terms"] + 8) == INVALID and policy(terms=PAT["w"] + 400) == INVALID
    assert policy(ws=None) == WORKSPACE and policy(ws_bytes=24) == WORKSPACE and policy(ws=PAT["ws"] + 8) == WORKSPACE
    assert policy(ws=PAT["d"]) == INVALID
    assert policy(adv=PAT["adv"] + 2) == ALIGN
    n = ctypes.c_size_t(1)
    lib = B.load_library()
    assert lib.muon_policy_loss_workspace_bytes(5, None) == INVALID
    assert lib.muon_policy_loss_workspace_bytes(-1, ctypes.byref(n)) == SHAPE
    assert lib.muon_policy_loss_workspace_bytes(100, ctypes.byref(n)) == 0 and n.value == 0


def test_preference_refusals():
    assert pref(tokens=-1) == SHAPE and pref(pairs=-1) == SHAPE and pref(pairs=(1 << 20) + 1) == SHAPE
    for v in (NAN, INF):
        assert pref(beta=v) == INVALID and pref(margin=v) == INVALID
    for v in (-0.1, 1.1, NAN):
        assert pref(smoothing=v) == INVALID
    assert pref(average=2) == INVALID
    for n in ("lp", "off", "loss"):
        assert pref(**{n: None}) == INVALID
    assert pref(off=PAT["off"] + 4) == ALIGN
    assert pref(d=PAT["ref"] + 4) == INVALID and pref(rew=PAT["w"]) == INVALID and pref(loss=PAT["off"]) == INVALID
    assert pref(d=PAT["valid"]) == INVALID
    assert pref(ws=None) == WORKSPACE and pref(ws_bytes=8) == WORKSPACE
    n = ctypes.c_size_t(1)
    lib = B.load_library()
    assert lib.muon_preference_loss_workspace_bytes(5, 1, None) == INVALID
    assert lib.muon_preference_loss_workspace_bytes(5, -1, ctypes.byref(n)) == SHAPE
    assert lib.muon_preference_loss_workspace_bytes(500, 30, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.muon_preference_loss_workspace_bytes(500, 3, ctypes.byref(n)) == 0 and n.value == 0


# ---- the binding -------------------------------------------------------------------

def _status(f, *a, **k):
    with pytest.raises(B.MuonError) as e:
        f(*a, **k)
    return e.value.status


def test_binding_rejects_heads_that_do_not_match():
    q, k, g = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16), torch.zeros(16)
    c = torch.zeros(9, 8)
    args = lambda **kw: [{**dict(q=q, k=k, gq=g, gk=g, c=c, s=c.clone(), qo=q.clone(), ko=k.clone()), **kw}[n]
                         for n in ("q", "k", "gq", "gk", "c", "s", "qo", "ko")]
    run = lambda **kw: _status(O.qk_norm_rope, *args(**{n: v for n, v in kw.items() if n != "positions"}),
                               **({"positions": kw["positions"]} if "positions" in kw else {}))
    assert run() == INVALID                                      # host tensors
    assert run(q=torch.zeros(16)) == SHAPE and run(q=torch.zeros(5, 4, 16)) == SHAPE
    assert run(k=torch.zeros(2, 5, 2, 8)) == SHAPE and run(k=k.bfloat16()) == DTYPE
    assert run(qo=q[:, :4]) == SHAPE and run(qo=q.bfloat16()) == DTYPE
    assert run(ko=None) == INVALID and run(k=None) == INVALID
    assert run(q=q.transpose(2, 3).contiguous().transpose(2, 3)) == INVALID   # dim is not contiguous
    assert run(gq=torch.zeros(15)) == SHAPE and run(gk=g.bfloat16()) == DTYPE
    assert run(c=None) == INVALID and run(s=torch.zeros(9, 4)) == SHAPE and run(c=c.double(), s=c.double()) == DTYPE
    assert run(c=torch.zeros(9, 16)[:, ::2], s=c) == INVALID
    for p, want in ((torch.zeros(5), DTYPE), (torch.zeros(2, 4, dtype=torch.int64), SHAPE),
                    (torch.zeros(3, 5, dtype=torch.int64), SHAPE), (torch.zeros(5, 2, dtype=torch.int64).t(), INVALID)):
        assert run(positions=p) == want
    z = lambda t: torch.zeros_like(t)
    assert _status(O.qk_norm_rope_backward, z(q), z(k), q, k, g, g, c, c, z(q), None) == INVALID
    assert _status(O.qk_norm_rope_backward, z(q), z(k), q, k, g, g, c, c, z(q), z(k), dgamma_q=g.bfloat16()) == DTYPE
    assert _status(O.qk_norm_rope_backward, z(q), z(k), q, k, g, g, c, c, z(q), z(k)) == INVALID


def test_binding_rejects_loss_arguments_that_do_not_match():
    x, t, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    assert _status(O.token_logp, x, t.int(), f, f) == DTYPE
    assert _status(O.token_logp, x, t[:3], f, f) == SHAPE
    assert _status(O.token_logp, x, t, f.double(), f) == DTYPE
    assert _status(O.token_logp, x.half(), t, f, f) == INVALID      # a host tensor before its type
    assert _status(O.token_logp, x, t, f, f) == INVALID
    assert _status(O.token_logp_backward, x, t, f, f, f, torch.zeros(4, 9)) == SHAPE
    assert _status(O.token_logp_backward, x, t, f, f, f[:3], x) == SHAPE
    one = torch.zeros(1)
    assert _status(O.policy_loss, f, f[:3], f, one) == SHAPE
    assert _status(O.policy_loss, f, f, f, one, weight=f.double()) == DTYPE
    assert _status(O.policy_loss, f, f, f, one, terms=torch.zeros(2)) == SHAPE
    assert _status(O.policy_loss, f, f, f, one) == INVALID
    off = torch.tensor([0, 2, 4])
    assert _status(O.preference_loss, f, off[:2], one) == SHAPE
    assert _status(O.preference_loss, f, off.int(), one) == DTYPE
    assert _status(O.preference_loss, f, off, one, weight=torch.zeros(2)) == SHAPE
    assert _status(O.preference_loss, f, off, one, rewards=torch.zeros(1)) == SHAPE
    assert _status(O.preference_loss, f, off, one, valid=torch.ones(4)) == DTYPE
    assert _status(O.preference_loss, f, off, one) == INVALID


def test_binding_rejects_tensors_of_two_devices(monkeypatch):
    """Every tensor's device is compared with the first one's (tensors whose device
    is faked: nothing is launched)."""
    class On(torch.Tensor):
        def get_device(self):
            return self.on

    def put(t, dev):
        t = t.as_subclass(On)
        t.on = dev
        return t

    monkeypatch.setattr(O, "_call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    heads, vec, words = lambda: torch.zeros(2, 5, 4, 16), lambda n: torch.zeros(n), lambda *s: torch.zeros(*s, dtype=torch.int64)
    calls = [
        (O.qk_norm_rope, [heads(), heads(), vec(16), vec(16), torch.zeros(9, 8), torch.zeros(9, 8), heads(), heads()],
         dict(positions=words(2, 5))),
        (O.qk_norm_rope_backward, [heads(), heads(), heads(), heads(), vec(16), vec(16), torch.zeros(9, 8),
                                   torch.zeros(9, 8), heads(), heads()],
         dict(positions=words(2, 5), dgamma_q=vec(16), dgamma_k=vec(16), workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
        (O.token_logp, [torch.zeros(4, 70000), words(4), vec(4), vec(4)], dict(workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
        (O.token_logp_backward, [torch.zeros(4, 8), words(4), vec(4), vec(4), vec(4), torch.zeros(4, 8)], {}),
        (O.policy_loss, [vec(5000), vec(5000), vec(5000), vec(1)],
         dict(ref_logp=vec(5000), weight=vec(5000), dlogp=vec(5000), dloss=vec(1), terms=vec(3),
              workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
        (O.preference_loss, [vec(500), words(61), vec(1)],
         dict(ref_logp=vec(500), valid=torch.zeros(500, dtype=torch.uint8), weight=vec(30), rewards=vec(60), dlogp=vec(500),
              dloss=vec(1), workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
    ]
    for f, args, kw in calls:
        count = len(args) + len(kw)
        for odd in range(count):
            a = [put(t, 1 if i == odd else 0) for i, t in enumerate(args)]
            k = {n: put(t, 1 if len(args) + i == odd else 0) for i, (n, t) in enumerate(kw.items())}
            assert _status(f, *a, **k) == INVALID, (f.__name__, odd)
        # host tensors
        assert _status(f, *args, **kw) == INVALID, f.__name__
