"""Argument checks of dn_accept_sampled, dn_rope_append, dn_head_norm and dn_residual_norm, on the host before anything is
enqueued (no GPU), and the frequencies that the binding makes."""

import math

import pytest
import torch

from deltanet_recurrent_state_gb300 import binding
from deltanet_recurrent_state_gb300 import build as dnbuild
from tests.test_abi import Bufs

OK, INVALID, UNSUPPORTED = binding.DN_OK, binding.DN_ERR_INVALID_ARG, binding.DN_ERR_UNSUPPORTED
F16, F32, BF16, E4M3 = binding.DN_F16, binding.DN_F32, binding.DN_BF16, binding.DN_E4M3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    dnbuild.build()
    return binding.load_library()


def filled(defaults, over):
    """`defaults` with `over`, where off_x is buffer x moved by some bytes; buffers are the Ellipsis values."""
    buf = Bufs()
    a = {x: buf() if y is ... else y for x, y in defaults.items()}
    for x, y in over.items():
        if x.startswith("off_"):
            a[x[4:]] = buf(offset=y)
        else:
            a[x] = y
    return list(a.values()) + [None]


SAMPLE = dict(B=2, T=3, V=100, dt=F16, logits=..., draft=..., uniform=..., temperature=..., top_k=..., top_p=..., min_p=..., target=...,
              accepted=..., logprob=..., ws=..., wsb=1 << 20)


@pytest.mark.parametrize("over,want", [
    (dict(B=-1), INVALID), (dict(T=0), INVALID), (dict(V=0), INVALID), (dict(dt=-1), INVALID), (dict(dt=4), INVALID), (dict(dt=E4M3), UNSUPPORTED),
    (dict(V=400001), UNSUPPORTED), (dict(B=1 << 20, T=1 << 10), INVALID), (dict(wsb=8), INVALID), (dict(ws=None), INVALID),
    (dict(off_logits=8), INVALID), (dict(off_ws=8), INVALID)]
    + [({x: None}, INVALID) for x in ("logits", "draft", "uniform", "temperature", "target", "accepted")]
    + [({"off_" + x: 2}, INVALID) for x in ("draft", "uniform", "temperature", "top_k", "top_p", "min_p", "target", "accepted", "logprob")])
def test_accept_sampled_rejects(lib, over, want):
    assert lib.dn_accept_sampled(*filled(SAMPLE, over)) == want


def test_accept_sampled_of_nothing_and_workspace_sizes(lib):
    assert lib.dn_accept_sampled(*filled(SAMPLE, dict(B=0))) == OK
    f = lib.dn_sample_workspace_bytes
    assert f(0, 1, 10) == f(1, 0, 10) == f(1, 1, 0) == f(1, 1, 400001) == f(1 << 20, 1 << 10, 10) == 0
    assert all(f(b, t, 1000) % 16 == 0 and f(b, t, 1000) >= 4 * (b + b * t) for b in (1, 3, 64) for t in (1, 16))


ROPE = dict(B=1, total=2, heads=1, group=2, D=64, rot=32, page=16, max_pages=1, pages=1, io=F16, cache=F16, inter=0, q=..., qs=128, k=..., ks=64,
            v=..., vs=64, positions=..., freqs=..., amplitude=1.0, qw=..., kw=..., eps=1e-6, start=..., kv=..., table=..., kc=..., vc=..., ke=..., ve=...,
            out=...)


@pytest.mark.parametrize("over,want", [
    (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(total=(1 << 28) + 1), INVALID), (dict(heads=0), INVALID), (dict(group=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=40), UNSUPPORTED), (dict(rot=80), UNSUPPORTED),
    (dict(rot=-16), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(io=F32, cache=F32), UNSUPPORTED), (dict(io=F16, cache=BF16), UNSUPPORTED),
    (dict(io=9), INVALID), (dict(max_pages=-1), INVALID), (dict(pages=-1), INVALID), (dict(qs=120), INVALID), (dict(qs=132), INVALID),
    (dict(ks=56), INVALID), (dict(vs=68), INVALID), (dict(amplitude=0.0), INVALID), (dict(amplitude=NAN), INVALID), (dict(amplitude=INF), INVALID),
    (dict(qw=None), INVALID), (dict(kw=None), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(group=1 << 18, qs=1 << 24), INVALID),
    (dict(group=1 << 19, qs=1 << 25), INVALID), (dict(total=1 << 28, group=128, qs=1 << 13), INVALID), (dict(cache=E4M3, ke=None), INVALID),
    (dict(cache=E4M3, off_ve=8), INVALID), (dict(off_positions=2), INVALID), (dict(off_freqs=4), INVALID), (dict(off_qw=8), INVALID),
    (dict(off_q=8), INVALID), (dict(off_out=8), INVALID), (dict(off_kc=8), INVALID), (dict(off_start=2), INVALID)]
    + [({x: None}, INVALID) for x in ("q", "k", "v", "freqs", "out", "start", "kv", "table", "kc", "vc")])
def test_rope_append_rejects(lib, over, want):
    if over.get("group") == 1 << 18:
        over = dict(over, D=64, total=1 << 20)  # (few enough elements a row, but too many warps)
    assert lib.dn_rope_append(*filled(ROPE, over)) == want


@pytest.mark.parametrize("over", [
    dict(heads=1 << 30, D=256, rot=256, group=(1 << 26) - 2, qs=1 << 40, ks=1 << 40, vs=1 << 40),
    dict(heads=1 << 30, D=256, rot=256, group=1 << 26, qs=0, ks=1 << 38, vs=1 << 38),
    dict(heads=(1 << 31) - 1, group=(1 << 31) - 1, qs=1 << 62, ks=1 << 62, vs=1 << 62), dict(heads=1 << 19, group=1, qs=1 << 25, ks=1 << 25, vs=1 << 25),
    dict(heads=1 << 9, group=1 << 10, qs=1 << 25, ks=1 << 15, vs=1 << 15)])
def test_rope_append_rejects_products_of_heads_past_its_bound(lib, over):
    """heads * group * D > 2^24, also where that product or the number of warps is small modulo 2^64."""
    for total in (1, 2):
        assert lib.dn_rope_append(*filled(ROPE, dict(over, total=total))) == INVALID


def test_rope_append_of_nothing(lib):
    assert lib.dn_rope_append(*filled(ROPE, dict(total=0))) == OK
    assert lib.dn_rope_append(*filled(ROPE, dict(B=0))) == OK


HEAD = dict(rows=2, heads=3, D=64, io=F16, order=0, act=2, x=..., xs=192, gate=..., gs=192, weight=..., eps=1e-6, out=...)


@pytest.mark.parametrize("over,want", [
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(D=32), UNSUPPORTED), (dict(io=E4M3), UNSUPPORTED), (dict(io=5), INVALID),
    (dict(order=3), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(xs=184), INVALID), (dict(xs=196), INVALID), (dict(gs=128), INVALID),
    (dict(io=F32, xs=198), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(order=1, gate=None), INVALID),
    (dict(order=2), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(off_x=8), INVALID), (dict(off_gate=8), INVALID),
    (dict(off_weight=8), INVALID), (dict(off_out=8), INVALID), (dict(heads=1 << 19, xs=1 << 25, gs=1 << 25), INVALID),
    (dict(rows=1 << 30, heads=4, xs=256, gs=256), INVALID),
])
def test_head_norm_rejects(lib, over, want):
    assert lib.dn_head_norm(*filled(HEAD, over)) == want


RES = dict(rows=2, C=64, io=F16, res=F16, act=1, y=..., ys=64, gate=..., gs=64, after=..., scale=1.0, residual=..., out_r=..., weight=..., eps=1e-6, out=...)


@pytest.mark.parametrize("over,want", [
    (dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(C=60), UNSUPPORTED), (dict(C=16392, ys=16392, gs=16392), UNSUPPORTED), (dict(io=E4M3), UNSUPPORTED),
    (dict(io=7), INVALID), (dict(res=BF16), UNSUPPORTED), (dict(res=7), INVALID), (dict(io=F32), UNSUPPORTED), (dict(act=5), INVALID), (dict(ys=56), INVALID),
    (dict(ys=68), INVALID), (dict(gs=32), INVALID), (dict(y=None), INVALID), (dict(y=None, gate=None), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(eps=-1.0), INVALID), (dict(residual=None), INVALID), (dict(out_r=None), INVALID), (dict(out=None), INVALID),
    (dict(off_y=8), INVALID), (dict(off_after=8), INVALID), (dict(off_residual=8), INVALID), (dict(off_out_r=8), INVALID), (dict(off_weight=8), INVALID),
])
def test_residual_norm_rejects(lib, over, want):
    assert lib.dn_residual_norm(*filled(RES, over)) == want


def test_norms_of_nothing(lib):
    assert lib.dn_head_norm(*filled(HEAD, dict(rows=0, x=None, out=None))) == OK
    assert lib.dn_residual_norm(*filled(RES, dict(rows=0, residual=None, out=None))) == OK


def turns_of(freqs):
    return [int(f) / 2.0 ** 64 for f in freqs]


def test_rope_freqs_on_the_ramp():
    """Pairs that turn 8.75, 16.5 and 24.25 times in the context are a quarter, a half and three quarters of the way, and those of 1 and 32 turns its ends."""
    for factor, context in ((4.0, 4096), (2.0, 1000)):
        for turns, way in ((8.75, 0.25), (16.5, 0.5), (24.25, 0.75), (1.0, 0.0), (32.0, 1.0), (0.5, 0.0), (40.0, 1.0)):
            base = (context / (2 * math.pi * turns)) ** 2  # pair 16 of 32 turns base^(-1/2) radians a token
            plain, _ = binding.rope_freqs(64, base=base, device="cpu")
            ramp, _ = binding.rope_freqs(64, base=base, scaling="ramp", factor=factor, context=context, device="cpu")
            assert abs(turns_of(plain)[16] * context - turns) < 1e-9
            assert abs(turns_of(ramp)[16] * context - turns * (way + (1 - way) / factor)) < 1e-9


def test_rope_freqs():
    freqs, amplitude = binding.rope_freqs(64, base=1e6, device="cpu")
    assert amplitude == 1.0 and freqs.dtype == torch.int64 and freqs.shape == (32,)
    plain = turns_of(freqs)
    for j, t in enumerate(plain):
        assert abs(t * 2 * math.pi - 1e6 ** (-2 * j / 64)) <= 1e-15
    linear, _ = binding.rope_freqs(64, base=1e6, scaling="linear", factor=4.0, device="cpu")
    assert all(abs(a * 4 - b) < 1e-15 for a, b in zip(turns_of(linear), plain))
    base, _ = binding.rope_freqs(64, base=1e6, scaling="base", factor=4.0, device="cpu")
    base = turns_of(base)
    assert base[0] == plain[0] and abs(base[-1] * 4 / plain[-1] - 1) < 1e-12 and all(b <= a for a, b in zip(plain, base))
    ramp, amplitude = binding.rope_freqs(64, base=1e6, scaling="ramp", factor=4.0, context=4096, device="cpu")
    assert abs(amplitude - (1 + 0.1 * math.log(4.0))) < 1e-12
    for a, b in zip(plain, turns_of(ramp)):
        if 4096 * a >= 32:
            assert b == a
        elif 4096 * a <= 1:
            assert abs(4 * b / a - 1) < 1e-6  # (a 64-bit fraction of a turn has fewer digits where it is small)
        else:
            assert a / 4 < b < a
    for bad in (dict(rot=7), dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, scaling="other"), dict(rot=0)):
        with pytest.raises(ValueError):
            binding.rope_freqs(**bad, device="cpu")
