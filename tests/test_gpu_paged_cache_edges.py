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


def put(s, x, c):
    """Replaces the pool of x by the 8-bit form of c."""
    codes, E = oracle.quantise(n64(c))
    s.d[x] = (torch.from_numpy(codes), torch.from_numpy(E))


@pytest.mark.parametrize("small", [4e-6, 4e-8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,ctx", [(40, 88), (300, 84)])
def test_small_rows_beside_a_large_one_that_is_not_seen(cuda, rows, ctx, D, small):
    """8 bits: a draft of 448 that only the last row sees takes nothing from rows of 4 * 10^-6 or 4 * 10^-8 in its tile.

    A tile's elements are on a grid of 2^-24 where its largest row ends at 448 * 2^7: with 448, off by at most
    2^-32. For the values that is the error of the output; for the keys, times scale * sum |q|, that of a score
    (relative, twice, that of a probability). q's elements below 2^-14 of the row's largest are off by 2^-25 of it.
    """
    s = Setup([rows], [rows + ctx], 1, D, 64, "bf16", "e4m3", seed=D, dirty=False)
    g = torch.Generator().manual_seed(rows)
    last = int(s.table[0, (rows + ctx - 1) // 64]), (rows + ctx - 1) % 64
    for x in "kv":
        c = (torch.randn(s.d[x][0].shape, generator=g) * small).bfloat16()
        c[last[0], :, last[1]] = 448.0
        put(s, x, c)
    s.q = (torch.randn(s.q.shape, generator=g) * 0.25 / (small * D ** 0.5)).bfloat16()
    out, lse = attend(s, scale=1.0)
    q, k, v = n64(s.q), s.values("k"), s.values("v")
    ref, rlse, weight, size = oracle.attn_paged(q, s.start.numpy(), s.kv, s.table.numpy(), k, v, 1.0)
    ds = 2 * (2.0 ** -24 * (D + 4) * size + 2.0 ** -22 * (1 + size) + 2.0 ** -32 * np.abs(q).sum(-1)
              + 2.0 ** -25 * np.abs(q).max(-1) * D * 5 * small)
    tol = (2.0 ** -11 + ds[..., None] + 2.0 ** -20) * weight + 2.0 ** -32 + 2.0 ** -8 * np.abs(ref)
    seen = slice(0, rows - 1)
    d = np.abs(n64(out) - ref)[seen]
    assert (d <= tol[seen]).all(), "out: %.3g of the bound" % (d / tol[seen]).max()
    dl = np.abs(n64(lse) - rlse)[seen]
    assert (dl <= ds[seen] + 2.0 ** -22 * (1 + np.abs(rlse[seen]))).all()


@pytest.mark.parametrize("size", [-100, -112, -122])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_smallest_values_of_bf16(cuda, rows, D, size):
    """Values of 2^-100 to 2^-122 in 8 bits come back with the precision of larger ones (bf16's grid ends at 2^-133)."""
    s = Setup([rows], [rows + 700], 1, D, 64, "bf16", "e4m3", seed=D, dirty=False)
    g = torch.Generator().manual_seed(rows)
    put(s, "v", (torch.randn(s.d["v"][0].shape, generator=g, dtype=torch.float64) * 2.0 ** size).bfloat16())
    out, lse = attend(s)
    q, k, v = n64(s.q), s.values("k"), s.values("v")
    ref, _, weight, x = oracle.attn_paged(q, s.start.numpy(), s.kv, s.table.numpy(), k, v, D ** -0.5)
    ds = 2 * (2.0 ** -24 * (D + 4) * x + 2.0 ** -22 * (1 + x))
    most = np.abs(v).max() * (rows + 700)
    tol = (2.0 ** -11 + ds[..., None] + 2.0 ** -20) * weight + 2.0 ** -25 * most + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    d = np.abs(n64(out) - ref)
    assert (d <= tol).all(), "out: %.3g of the bound" % (d / tol).max()


# ---- windows and lengths ------------------------------------------------------------------------

@pytest.mark.parametrize("io,cache", [("f16", "io"), ("bf16", "io"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kv,group,window", [([1], [1000], 1, 100), ([16, 3], [900, 150], 6, 77), ([150, 40], [410, 700], 2, 100),
                                              ([300], [1200], 1, 513)])
def test_what_lies_before_the_window_may_be_anything(cuda, n, kv, group, window, D, io, cache):
    s = Setup(n, kv, 2, D, 64, io, cache, seed=window, group=group)
    for b in range(len(n)):
        for j in range(max(0, kv[b] - n[b] - window + 1)):
            at = int(s.table[b, j // 64]), j % 64
            s.own[at] = False
            for x in "kv":
                c, E = s.d[x]
                c[at[0], :, at[1]] = float("nan") if E is None else 0x7F
                if E is not None:
                    E[at[0], :, at[1]] = 255
    check_attn(s, *attend(s, window=window), window=window)


@pytest.mark.parametrize("cache", ["io", "e4m3"])
def test_append_and_gather_clamp_the_length(cuda, cache):
    """kv_len above the most tokens counts as that, as for the attention."""
    s = Setup([2], [128], 1, 64, 128, "f16", cache, dirty=False)
    w = s.where()
    table = torch.full((1, 1 << 23), -1, dtype=torch.int32, device="cuda")  # 2^30 positions
    table[0, -1] = s.table[0, 0]
    k, v = (x.cuda() for x in s.new)
    a, b = [t if t is None else t.clone() for t in w], [t if t is None else t.clone() for t in w]
    a[2] = b[2] = table
    a[1] = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    b[1] = torch.tensor([(1 << 30) + 1], dtype=torch.int32, device="cuda")
    dn.dn_kv_append(k, v, *a)
    dn.dn_kv_append(k, v, *b)
    dn.dn_kv_append(k, v, *w)  # the same rows of the page, by a short table
    for i in (3, 4):
        assert torch.equal(a[i].view(torch.uint8), b[i].view(torch.uint8)) and torch.equal(a[i].view(torch.uint8), w[i].view(torch.uint8))
    got, want = [[torch.full_like(x, float("nan")) for x in (k, v)] for _ in range(2)]
    dn.dn_kv_gather(*b, *got)
    dn.dn_kv_gather(*w, *want)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_gather_of_no_request_gives_zeros(cuda):
    s = Setup([2], [5], 1, 64, 16, "f16", "io", dirty=False)
    w = s.where()
    w[0], w[1] = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    w[2] = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    k, v = (torch.full((3, 1, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    dn.dn_kv_gather(*w, k, v)
    assert (k == 0).all() and (v == 0).all()


# ---- the binding --------------------------------------------------------------------------------

def test_a_cache_without_heads_is_refused(cuda):
    s = Setup([2], [5], 1, 64, 16, "f16", "io", dirty=False)
    w = s.where()
    w[3], w[4] = w[3][:, :0].contiguous(), w[4][:, :0].contiguous()
    with pytest.raises(ValueError):
        dn.dn_attn_paged(s.q.cuda(), *w)


def test_windows_past_32_bits(cuda):
    s = Setup([3], [200], 1, 64, 16, "f16", "io", dirty=False)
    w, q = s.where(), s.q.cuda()
    want = dn.dn_attn_paged(q, *w)
    for window in ((1 << 32) + 5, 1 << 31, 1 << 64):
        got = dn.dn_attn_paged(q, *w, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for window in (-1, -(1 << 32) + 5):
        with pytest.raises(dn.DnError):
            dn.dn_attn_paged(q, *w, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_many_improbable_tokens_in_fp16(cuda, rows, D):
    """Tokens whose probabilities are below fp16's smallest number each, and count together.

    Every 2,000th key scores 17.5 above the others (by a product of 1 and 17.5, exact), with a value of 0 against 64:
    out = 64 r / (1 + r) with r = 1,999 e^-17.5. Bounds: 2^-11 for a probability (2^-7 of it on the finest grid), 2^-11
    for the output and its grid of 2^-24, and 2^-18 for the exponential and the sums.
    """
    heads, page, kv = 160, 128, 16000
    pages = kv // page
    k = torch.zeros((pages, heads, page, D), dtype=torch.float16, device="cuda")
    v = torch.full_like(k, 64.0)
    hot = torch.arange(0, kv, 2000, device="cuda") + 1000
    k[hot // page, :, hot % page, 0], v[hot // page, :, hot % page] = 17.5, 0.0
    q = torch.zeros((rows, heads, D), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, _ = dn.dn_attn_paged(q, one(0, rows), one(kv), table, k, v, scale=1.0)
    # rows see kv - rows + 1 + i tokens: all hot ones (the last at 15,000), fewer others
    others = torch.arange(kv - rows + 1, kv + 1, dtype=torch.float64) - 8
    r = others / 8 * torch.exp(torch.tensor(-17.5, dtype=torch.float64))
    ref = (64 * r / (1 + r))[:, None, None]
    d = (out.double().cpu() - ref).abs()
    assert (d <= (2.0 ** -7 + 2.0 ** -11 + 2.0 ** -18) * ref + 2.0 ** -25).all()


# ---- repeats ------------------------------------------------------------------------------------

@pytest.mark.parametrize("io,cache", [("f16", "io"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,group", [(1, 4), (40, 4), (300, 4), (16, 5), (1, 129)])
def test_every_output_is_written_alike_again(cuda, rows, group, D, io, cache):
    """Ranges that are joined, into outputs of NaN, with a workspace of ones (NaN too) and of zeros."""
    s = Setup([rows, 5, 1], [3000, 900, 2500], 2, D, 64, io, cache, group=group)
    w, q = s.where(), s.q.cuda()
    got = []
    for fill in (255, 0):
        ws = dn.attn_workspace(q, w[3], w[2]).fill_(fill)
        out = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        got.append(dn.dn_attn_paged(q, *w, out=out, lse=lse, workspace=ws))
    assert dn.dn_attn_wait_timeouts() == 0
    assert all(torch.isfinite(t).all() for t in got[0])
    assert all(torch.equal(a, b) for a, b in zip(*got))
