"""The paged cache on the GPU where it can go wrong: groups, extreme sizes of values, windows, streams, lengths.

The attention is held to the bounds that tests/test_gpu_paged_cache.py derives, unless a test states its own.
Outputs are filled with NaN before every call, so that what a call leaves unwritten shows.
"""

import numpy as np
import pytest
import torch

import oracle
from deltanet_recurrent_state_gb300 import binding as dn
from tests.test_gpu_paged_cache import E4M3, Setup, check_attn, n64

pytestmark = pytest.mark.gpu


def attend(s, window=0, scale=None, where=None):
    out = torch.full(s.q.shape, float("nan"), dtype=s.io, device="cuda")
    lse = torch.full(s.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
    dn.dn_attn_paged(s.q.cuda(), *(where or s.where()), window=window, scale=scale, out=out, lse=lse)
    assert dn.dn_attn_wait_timeouts() == 0
    return out, lse


# ---- groups -------------------------------------------------------------------------------------

@pytest.mark.parametrize("io,cache", [("f16", "io"), ("bf16", "io"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [5, 11, 33, 128])
def test_groups_of_many_heads_in_tiles(cuda, group, D, io, cache):
    """D = 256 with 5, 11 or 33 heads a key head: tiles of an odd number of rows, cut into ranges and joined."""
    s = Setup([16, 3], [2000, 700], 1, D, 64, io, cache, seed=group, group=group)
    check_attn(s, *attend(s))


@pytest.mark.parametrize("cache", ["io", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kv,group", [([1], [900], 129), ([2, 0, 3], [40, 9, 700], 160)])
def test_groups_of_more_heads_than_a_tile_has_rows(cuda, n, kv, group, D, cache):
    s = Setup(n, kv, 1, D, 32, "f16", cache, seed=group, group=group)
    check_attn(s, *attend(s))
    check_attn(s, *attend(s, window=70), window=70)


# ---- extreme sizes ------------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [None, 2.0 ** -30])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [2, 40, 300])
def test_queries_and_keys_of_zero(cuda, rows, D, scale):
    """Scores of 0 under a mask: the mean of the values that a row sees, and the log of their number."""
    s = Setup([rows], [rows + 150], 1, D, 64, "bf16", "e4m3", seed=rows)
    codes, E = s.d["k"]
    held = s.own[:, None, :].expand(E.shape)
    codes[held], E[held] = 0, 0
    s.q[:] = 0
    s.q[rows // 2, :, 0] = 2.0 ** -120
    check_attn(s, *attend(s, scale=scale), scale=scale)


# ---- streams ------------------------------------------------------------------------------------

def slow(ms):
    torch.cuda._sleep(int(ms * 1.5e6))


def test_workspace_of_a_call_on_another_stream(cuda):
    """What the call allocated for itself is not handed out again while the call is still waiting to run."""
    s = Setup([16], [3000], 2, 128, 64, "f16", "io", group=3)
    w, q = s.where(), s.q.cuda()
    want = [t.clone() for t in dn.dn_attn_paged(q, *w)]
    bytes_ = dn.attn_workspace(q, w[3], w[2]).numel()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            slow(50)
        out, lse = dn.dn_attn_paged(q, *w, stream=stream)
        mine = [torch.full((bytes_,), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        assert all((m == 7).all() for m in mine)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        del mine


def test_outputs_of_a_call_on_another_stream(cuda):
    """Outputs do not take memory that work queued on the current stream still uses."""
    s = Setup([16], [300], 2, 128, 64, "f16", "io", group=3)
    w, q = s.where(), s.q.cuda()
    ws = dn.attn_workspace(q, w[3], w[2])
    dn.dn_attn_paged(q, *w, workspace=ws)
    side = torch.cuda.Stream()
    copy = torch.empty_like(q)
    old = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    slow(50)
    copy.copy_(old)
    del old
    out, _ = dn.dn_attn_paged(q, *w, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert (copy == 7).all()


def test_accept_on_another_stream(cuda):
    """The same of dn_accept_greedy, whose workspace has to be zero when the call runs."""
    logits = torch.randn((2, 16, 4096), device="cuda").half()
    drafts = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    want = [t.clone() for t in dn.dn_accept_greedy(logits, drafts)]
    n = dn.accept_workspace(2, 16, 4096, logits.device).numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        slow(50)
    got = dn.dn_accept_greedy(logits, drafts, stream=side)
    mine = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all((m == 255).all() for m in mine)
