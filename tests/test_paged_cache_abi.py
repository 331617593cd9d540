"""Argument checks of the paged-cache entry points, on the host before anything is enqueued (no GPU)."""

import pytest

from deltanet_recurrent_state_gb300 import binding
from deltanet_recurrent_state_gb300 import build as dnbuild
from tests.test_abi import Bufs

OK, INVALID, UNSUPPORTED = binding.DN_OK, binding.DN_ERR_INVALID_ARG, binding.DN_ERR_UNSUPPORTED
F16, F32, BF16, E4M3 = binding.DN_F16, binding.DN_F32, binding.DN_BF16, binding.DN_E4M3


@pytest.fixture(scope="module")
def lib():
    dnbuild.build()
    return binding.load_library()


def args(call, **over):
    buf = Bufs()
    a = dict(B=1, total=2, heads=1, group=1, D=64, page=16, max_pages=1, pages=1, io=F16, cache=F16, k=buf(), v=buf(), q=buf(),
             ks=64, vs=64, qs=64, start=buf(), kv=buf(), table=buf(), kc=buf(), vc=buf(), ke=buf(), ve=buf(), scale=0.125,
             window=0, out=buf(), lse=buf(), ws=buf(), wsb=1 << 40)
    for x, y in over.items():
        if x.startswith("off_"):
            a[x[4:]] = buf(offset=y)
        else:
            a[x] = y
    head = [a[x] for x in ("B", "total", "heads")]
    tail = [a[x] for x in ("D", "page", "max_pages", "pages", "io", "cache")]
    where = [a[x] for x in ("start", "kv", "table", "kc", "vc", "ke", "ve")]
    if call == "append":
        return head + tail + [a[x] for x in ("k", "v", "ks", "vs")] + where + [None]
    if call == "gather":
        return head + tail + where + [a["k"], a["v"], None]
    return head + [a["group"]] + tail + [a["q"], a["qs"]] + where + [a[x] for x in ("scale", "window", "out", "lse", "ws", "wsb")] + [None]


NAMES = {"append": "dn_kv_append", "gather": "dn_kv_gather", "attn": "dn_attn_paged"}


@pytest.mark.parametrize("call", NAMES)
@pytest.mark.parametrize("over,want", [
    (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(total=(1 << 28) + 1), INVALID), (dict(heads=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=32), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=256), UNSUPPORTED), (dict(io=F32, cache=F32), UNSUPPORTED), (dict(io=E4M3, cache=E4M3), UNSUPPORTED),
    (dict(io=F16, cache=BF16), UNSUPPORTED), (dict(io=BF16, cache=F16), UNSUPPORTED), (dict(io=7), INVALID), (dict(cache=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(pages=-1), INVALID), (dict(max_pages=(1 << 26) + 1), INVALID),
    (dict(start=None), INVALID), (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(cache=E4M3, ke=None), INVALID), (dict(cache=E4M3, ve=None), INVALID),
    (dict(off_start=2), INVALID), (dict(off_kv=1), INVALID), (dict(off_table=2), INVALID), (dict(off_kc=8), INVALID),
    (dict(off_vc=4), INVALID), (dict(cache=E4M3, off_ke=8), INVALID),
])
def test_every_call_rejects(lib, call, over, want):
    assert getattr(lib, NAMES[call])(*args(call, **over)) == want


@pytest.mark.parametrize("call,over", [
    ("append", dict(k=None)), ("append", dict(v=None)), ("append", dict(off_k=8)), ("append", dict(ks=63)), ("append", dict(ks=68)),
    ("append", dict(vs=56)), ("append", dict(heads=1 << 20, ks=1 << 27, vs=1 << 27)), ("gather", dict(k=None)), ("gather", dict(off_v=8)),
    ("attn", dict(group=0)), ("attn", dict(window=-1)), ("attn", dict(scale=0.0)), ("attn", dict(scale=-0.5)),
    ("attn", dict(scale=float("inf"))), ("attn", dict(scale=float("nan"))), ("attn", dict(q=None)), ("attn", dict(out=None)),
    ("attn", dict(ws=None)), ("attn", dict(off_q=8)), ("attn", dict(off_out=2)), ("attn", dict(off_lse=2)), ("attn", dict(off_ws=8)),
    ("attn", dict(wsb=1024)), ("attn", dict(qs=32)), ("attn", dict(qs=68)), ("attn", dict(group=1 << 21, qs=1 << 28)),
])
def test_one_call_rejects(lib, call, over):
    assert getattr(lib, NAMES[call])(*args(call, **over)) == INVALID


@pytest.mark.parametrize("call", NAMES)
def test_nothing_to_do_is_ok(lib, call):
    assert getattr(lib, NAMES[call])(*args(call, total=0)) == OK


def test_workspace_sizes(lib):
    f = lib.dn_attn_workspace_bytes
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, 0, 64), (1, 1, 1, 1, 80)):
        assert f(*bad) == 0
    assert 0 < f(1, 1, 4, 6, 256) < 1 << 28 and f(64, 25000, 8, 4, 128) < 1 << 28
    assert all(f(b, t, 4, 6, 256) % 16 == 0 for b in (1, 64) for t in (1, 16, 2048))
