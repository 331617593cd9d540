"""The paged cache on the GPU against the oracle: dn_kv_append, dn_kv_gather, dn_attn_paged.

Tolerances of the attention, from its arithmetic (u = half a unit in the last place, relative):
  * scores: products of 16-bit values are exact in 32 bits and are summed in 32 bits, at worst
    2^-24 (D + 4) times sum |q k| (`size`); the exponential adds 2^-22;
    so a probability is off by at most ds = 2 (2^-24 (D + 4) size + 2^-22 (1 + |x|)) relative, |x| <= size;
  * probabilities are rounded to 16 bits before they meet the values: u_p = 2^-11 (fp16, and 8-bit caches)
    or 2^-8 (bf16: 7 fraction bits, so half a unit is 2^-8 at the bottom of a binade);
  * fp16 probabilities below 2^-14 are on a grid of 2^-24: at most 2^-25 |v| each, over at most kv_len tokens,
    against a sum of at least 1;
  * sums and joins in 32 bits: 2^-20 of the weighted |v|;
  * the output's own rounding u_o |out|, and 2^-25 below fp16's normal range.
So |out - ref| <= (u_p + ds + 2^-20) weight + 2^-25 sum |v| + u_o |ref| + 2^-25, element by element, and
|lse - ref| <= ds + 2^-22 (1 + |ref|).
"""

import numpy as np
import pytest
import torch

import oracle
from deltanet_recurrent_state_gb300 import binding as dn

pytestmark = pytest.mark.gpu

IO = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def n64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """A pool with requests' pages in random order; unowned pages and rows past kv_len hold NaN."""

    def __init__(self, n, kv, heads, D, page, io, cache, seed=0, group=1, spare=3, dirty=True, extra_table=1):
        g = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.io, self.cache, self.page = n, kv, IO[io], cache, page
        B = len(n)
        used = [-(-max(x, 0) // page) for x in kv]
        pages = sum(used) + spare
        order = torch.randperm(pages, generator=g)
        width = max(used + [0]) + extra_table
        table = torch.full((B, width), -1, dtype=torch.int32)
        own = torch.zeros((pages, page), dtype=torch.bool)
        at = 0
        for b in range(B):
            table[b, :used[b]] = order[at:at + used[b]].int()
            at += used[b]
            for j in range(max(kv[b], 0)):
                own[table[b, j // page], j % page] = True
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
        self.kv_len = torch.tensor(kv, dtype=torch.int32)
        self.table, self.own, self.total = table, own, sum(n)
        self.d = {}
        for x in "kv":
            size = torch.exp(torch.randn((pages, heads, page, 1), generator=g))
            c = (torch.randn((pages, heads, page, D), generator=g) * size).to(self.io)
            if cache == "e4m3":
                codes, E = oracle.quantise(n64(c))
                codes, E = torch.from_numpy(codes), torch.from_numpy(E)
                if dirty:
                    hole = ~own[:, None, :].expand(pages, heads, page)
                    codes[hole] = 0x7F
                    E[hole] = 255
                self.d[x] = (codes, E)
            else:
                if dirty:
                    c[~own[:, None, :].expand(pages, heads, page)] = float("nan")
                self.d[x] = (c, None)
        self.q = torch.randn((self.total, heads * group, D), generator=g).to(self.io)
        self.new = [(torch.randn((self.total, heads, D), generator=g) * torch.exp(torch.randn((self.total, heads, 1), generator=g))).to(self.io)
                    for _ in range(2)]

    def values(self, x):
        c, E = self.d[x]
        v = n64(c) if E is None else oracle.values(c.numpy(), E.numpy())
        return np.where(self.own[:, None, :, None].numpy(), v, 0.0)

    def where(self):
        k, v = self.d["k"], self.d["v"]
        view = lambda c, E: c.cuda() if E is None else c.cuda().view(E4M3)  # noqa: E731
        cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
        return [self.start.cuda(), self.kv_len.cuda(), self.table.cuda(), view(*k), view(*v), cuda(k[1]), cuda(v[1])]


def check_attn(s, out, lse, window=0, scale=None, q=None):
    q = n64(s.q if q is None else q)
    D, heads = q.shape[2], q.shape[1]
    scale = D ** -0.5 if scale is None else scale
    k, v = s.values("k"), s.values("v")
    ref, rlse, weight, size = oracle.attn_paged(q, s.start.numpy(), s.kv, s.table.numpy(), k, v, scale, window)
    u_p = 2.0 ** -8 if s.io == torch.bfloat16 and s.cache == "io" else 2.0 ** -11
    u_o = 2.0 ** -8 if s.io == torch.bfloat16 else 2.0 ** -11
    ds = 2 * (2.0 ** -24 * (D + 4) * size + 2.0 ** -22 * (1 + size))
    most = np.abs(v).max() * max(s.kv + [1])
    tol = (u_p + ds[..., None] + 2.0 ** -20) * weight + 2.0 ** -25 * most + u_o * np.abs(ref) + 2.0 ** -25
    d = np.abs(n64(out) - ref)
    assert np.isfinite(n64(out)).all()
    assert (d <= tol).all(), "out: %.3g of the bound at %s" % ((d / tol).max(), np.unravel_index((d / tol).argmax(), d.shape))
    empty = np.isneginf(rlse)
    got = n64(lse)
    assert (np.isneginf(got) == empty).all() and (n64(out)[empty] == 0).all()
    dl, tl = np.abs(got[~empty] - rlse[~empty]), ds[~empty] + 2.0 ** -22 * (1 + np.abs(rlse[~empty]))
    assert (dl <= tl).all(), "lse: %.3g of the bound" % (dl / tl).max()


def check_attn_some(s, out, lse, heads=(0, 17, 39), window=0):
    """check_attn on some of the heads (of group 1): the oracle is slow on large cases."""
    part = Setup.__new__(Setup)
    part.__dict__ = dict(s.__dict__)
    part.d = {x: (c[:, heads], None if E is None else E[:, heads]) for x, (c, E) in s.d.items()}
    part.q = s.q[:, heads]
    check_attn(part, out[:, heads], lse[:, heads], window)


# ---- append and gather ------------------------------------------------------------------------

SHAPES = [  # n, kv, heads, D, page
    ([1], [1], 1, 64, 16),
    ([16], [40], 4, 256, 64),
    ([3, 0, 17, 1], [3, 9, 33, 128], 3, 128, 32),
    ([5, 70], [90, 70], 8, 64, 128),
    ([2, 4, 1], [1, -7, 500], 5, 256, 16),
]


@pytest.mark.parametrize("cache", ["io", "e4m3"])
@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("n,kv,heads,D,page", SHAPES)
def test_append_then_gather(cuda, n, kv, heads, D, page, io, cache):
    s = Setup(n, kv, heads, D, page, io, cache, seed=D + page, dirty=False)
    w = s.where()
    new = [x.cuda() for x in s.new]
    dn.dn_kv_append(*new, *w)
    start, table = s.start.numpy(), s.table.numpy()
    for x, rows, got, E in zip("kv", s.new, w[3:5], w[5:7]):
        old = s.d[x]
        if cache == "io":
            assert np.array_equal(n64(got), oracle.kv_append(n64(rows), start, kv, table, n64(old[0])))
        else:
            codes, exps = oracle.quantise(n64(rows))
            assert np.array_equal(got.view(torch.uint8).cpu().numpy(), oracle.kv_append(codes, start, kv, table, old[0].numpy()))
            assert np.array_equal(E.cpu().numpy(), oracle.kv_append(exps, start, kv, table, old[1].numpy()))
    k, v = (torch.full_like(x, float("nan")) for x in new)
    dn.dn_kv_gather(*w, k, v)
    for got, c, E in zip((k, v), w[3:5], w[5:7]):
        held = n64(c) if E is None else oracle.values(c.view(torch.uint8).cpu().numpy(), E.cpu().numpy())
        want = torch.from_numpy(oracle.kv_gather(s.total, start, kv, table, held)).to(s.io)
        assert torch.equal(got.cpu(), want)


def test_append_takes_slices_of_a_projection(cuda):
    s = Setup([7, 2], [20, 2], 3, 64, 16, "f16", "io", dirty=False)
    a, b = s.where(), s.where()
    k, v = (x.cuda() for x in s.new)
    wide = torch.randn((s.total, 11, 64), device="cuda").half()
    wide[:, 2:5], wide[:, 8:11] = k, v
    dn.dn_kv_append(k, v, *a)
    dn.dn_kv_append(wide[:, 2:5], wide[:, 8:11], *b)
    assert all(torch.equal(x, y) for x, y in zip(a[3:5], b[3:5]))


def test_extreme_rows_in_8_bits(cuda):
    """Largest, smallest, infinite and NaN values of both types."""
    for io, big, tiny in (("f16", 65504.0, 2.0 ** -24), ("bf16", 3.3895313892515355e38, 2.0 ** -133)):
        s = Setup([6], [6], 1, 64, 16, io, "e4m3", dirty=False)
        x = torch.zeros((6, 1, 64))
        x[0, 0, 3], x[1, 0, 5] = big, -tiny
        x[2, 0, :2] = torch.tensor([float("nan"), 3.0])
        x[3, 0, :3] = torch.tensor([float("inf"), -float("inf"), 1.0])
        x[4] = torch.linspace(-1, 1, 64)
        x = x.to(s.io)
        w = s.where()
        dn.dn_kv_append(x.cuda(), x.cuda(), *w)
        k, v = torch.empty((6, 1, 64), dtype=s.io, device="cuda"), torch.empty((6, 1, 64), dtype=s.io, device="cuda")
        dn.dn_kv_gather(*w, k, v)
        got, xx = n64(k)[:, 0], n64(x)[:, 0]
        assert torch.equal(k.nan_to_num(7.0), v.nan_to_num(7.0))
        assert np.isfinite(got[0]).all() and abs(got[0, 3] - xx[0, 3]) <= xx[0, 3] / 16 and (got[0, :3] == 0).all()
        # fp16's smallest value is kept; bf16's is below 2^-127 times the smallest e4m3 step's reach only by its own grid
        assert abs(got[1, 5] - xx[1, 5]) <= abs(xx[1, 5]) / 16
        assert np.isnan(got[2, 0]) and got[2, 1] == 3.0
        assert got[3, 0] > 1e4 and got[3, 1] < -1e4 and np.isfinite(got[3]).all()
        assert np.abs(got[4] - xx[4]).max() <= 1 / 16 and (got[5] == 0).all()


def test_pages_that_are_not_there(cuda):
    s = Setup([40], [100], 2, 64, 16, "f16", "io", dirty=False)
    s.table[0, 5], s.table[0, 4] = 10 ** 6, -5
    w = s.where()
    before = w[3].clone()
    dn.dn_kv_append(*(x.cuda() for x in s.new), *w)
    start, table = s.start.numpy(), s.table.numpy()
    assert np.array_equal(n64(w[3]), oracle.kv_append(n64(s.new[0]), start, s.kv, table, n64(before)))
    k, v = (torch.empty((40, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    dn.dn_kv_gather(*w, k, v)
    assert np.array_equal(n64(k), oracle.kv_gather(40, start, s.kv, table, n64(w[3])))
    assert (k[4:20] == 0).all()  # positions 64 .. 79 of 60 .. 99


def test_rows_of_no_request_are_zeros(cuda):
    s = Setup([4], [4], 1, 64, 16, "f16", "io", dirty=False)
    s.start[:] = torch.tensor([1, 3])
    s.kv_len[:] = 2
    w = s.where()
    k, v = (torch.full((4, 1, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    dn.dn_kv_gather(*w, k, v)
    assert (k[0] == 0).all() and (k[3] == 0).all() and torch.equal(k[1:3, 0], w[3][s.table[0, 0], 0, :2])


# ---- attention --------------------------------------------------------------------------------

ATTN = [  # n, kv, key heads, group, D, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1000], 4, 6, 256, 64, 0),            # one token, cut into ranges
    ([16], [1500], 2, 6, 256, 64, 0),           # a verify block
    ([4, 4, 4, 4, 4], [300, 4, 77, 128, 1], 3, 4, 128, 64, 0),   # batch; the last has rows that see nothing
    ([1, 1, 1], [700, 0, 33], 8, 4, 128, 16, 0),  # a request with nothing cached
    ([2, 0, 3, 130], [40, 12, 3, 131], 2, 3, 64, 32, 0),
    ([33], [33], 1, 7, 128, 128, 0),            # a whole short prompt, odd group
    ([150, 3], [410, 700], 2, 8, 64, 32, 100),  # window
    ([5], [260], 1, 4, 128, 16, 1),             # a window of the token itself
    ([300], [555], 1, 2, 128, 16, 0),           # a chunk
    ([70], [200], 2, 1, 256, 32, 37),
    ([9, 40], [2, 30], 2, 5, 64, 16, 0),        # more new tokens than cached ones
]


@pytest.mark.parametrize("io,cache", [("f16", "io"), ("bf16", "io"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("n,kv,heads,group,D,page,window", ATTN)
def test_attention(cuda, n, kv, heads, group, D, page, window, io, cache):
    s = Setup(n, kv, heads, D, page, io, cache, seed=sum(n) + D, group=group)
    out = torch.full(s.q.shape, float("nan"), dtype=s.io, device="cuda")
    out, lse = dn.dn_attn_paged(s.q.cuda(), *s.where(), window=window, out=out)
    check_attn(s, out, lse, window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 12, 20, 96, 600])
def test_attention_of_long_caches(cuda, D, rows):
    """Many ranges of one tile, joined; values of very different sizes in the 8-bit cache."""
    s = Setup([rows], [6000], 1, D, 64, "f16", "e4m3", seed=rows, group=1)
    out, lse = dn.dn_attn_paged(s.q.cuda(), *s.where())
    check_attn(s, out, lse)


@pytest.mark.parametrize("io,cache", [("f16", "io"), ("bf16", "io"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,kv", [(40, 2700), (200, 1500), (300, 2600)])
def test_attention_of_many_tiles_in_one_unit(cuda, D, rows, kv, io, cache):
    """Enough heads that nothing is cut, and enough tokens that every ring goes round several times."""
    s = Setup([rows], [kv], 40, D, 128, io, cache, seed=rows, group=1)
    out, lse = dn.dn_attn_paged(s.q.cuda(), *s.where())
    check_attn_some(s, out, lse)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_attention_repeats_bit_for_bit(cuda, rows):
    s = Setup([rows, 5, 1], [5000, 900, 2500], 2, 128, 64, "bf16", "io", group=4)
    w, q = s.where(), s.q.cuda()
    ws = dn.attn_workspace(q, w[3], w[2])
    first = [t.clone() for t in dn.dn_attn_paged(q, *w, workspace=ws)]
    ws.fill_(255)
    again = dn.dn_attn_paged(q, *w, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("rows", [2, 100])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_a_slice_of_a_projection(cuda, rows, D):
    s = Setup([rows], [rows + 50], 2, D, 16, "f16", "io", group=2)
    wide = torch.randn((rows, 9, D), device="cuda").half()
    wide[:, 3:7] = s.q.cuda()
    w = s.where()
    a, b = dn.dn_attn_paged(wide[:, 3:7], *w), dn.dn_attn_paged(s.q.cuda(), *w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows,D", [(1, 128), (64, 128), (64, 256)])
@pytest.mark.parametrize("cache", ["io", "e4m3"])
def test_attention_reads_missing_pages_as_zeros(cuda, rows, D, cache):
    s = Setup([rows], [400], 1, D, 16, "f16", cache, group=1)
    holes = s.table[0, [3, 20]].clone()
    s.table[0, 3], s.table[0, 20] = 10 ** 6, -5
    s.own[holes.long()] = False  # (the oracle reads zeros there by the table)
    out, lse = dn.dn_attn_paged(s.q.cuda(), *s.where())
    check_attn(s, out, lse)


@pytest.mark.parametrize("rows,D", [(1, 128), (80, 128), (80, 64), (80, 256)])
def test_attention_of_very_different_scores(cuda, rows, D):
    """Scores of hundreds: the running maximum grows and falls far; values of very different sizes."""
    s = Setup([rows], [900], 1, D, 64, "f16", "e4m3", group=1, seed=5)
    q = (s.q.float() * 30).half()
    out, lse = dn.dn_attn_paged(q.cuda(), *s.where())
    check_attn(s, out, lse, q=q)


@pytest.mark.parametrize("rows", [1, 64])
def test_attention_in_a_pool_past_32_bits(cuda, rows):
    """Pages beyond 2^31 elements and 2^32 bytes of the pool."""
    D, heads, page = 128, 8, 128
    pages = (1 << 32) // (D * heads * page) + 8  # 2^32 elements: 8 GiB a pool
    s = Setup([rows], [300], heads, D, page, "f16", "io", group=1, dirty=False)
    w = s.where()
    pools = []
    for c in w[3:5]:
        big = torch.empty((pages, heads, page, D), dtype=torch.float16, device="cuda")
        big[-c.shape[0]:] = c
        pools.append(big)
    table = torch.where(w[2] >= 0, w[2] + pages - w[3].shape[0], w[2])
    out, lse = dn.dn_attn_paged(s.q.cuda(), w[0], w[1], table, *pools)
    check_attn(s, out, lse)
    dn.dn_kv_append(*(x.cuda() for x in s.new), w[0], w[1], table, *pools)
    k, v = (torch.empty_like(x.cuda()) for x in s.new)
    dn.dn_kv_gather(w[0], w[1], table, *pools, None, None, k, v)
    assert torch.equal(k.cpu(), s.new[0]) and torch.equal(v.cpu(), s.new[1])


def test_on_another_stream_and_in_a_graph(cuda):
    s = Setup([16, 3], [700, 90], 2, 128, 64, "f16", "e4m3", group=3)
    w, q = s.where(), s.q.cuda()
    want = [t.clone() for t in dn.dn_attn_paged(q, *w)]
    ws = dn.attn_workspace(q, w[3], w[2])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dn.dn_attn_paged(q, *w, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    k, v = (x.cuda() for x in s.new)
    with torch.cuda.graph(graph):
        dn.dn_kv_append(k, v, *w)
        dn.dn_attn_paged(q, *w, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    again = dn.dn_attn_paged(q, *w)
    assert torch.equal(out, again[0]) and not torch.equal(out, want[0])


def test_empty_calls(cuda):
    s = Setup([2], [5], 1, 64, 16, "f16", "io", dirty=False)
    w = s.where()
    none = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    w[0] = torch.zeros(2, dtype=torch.int32, device="cuda")
    dn.dn_kv_append(none, none, *w)
    dn.dn_kv_gather(*w, none, none)
    out, lse = dn.dn_attn_paged(none, *w)
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1)
    # no pages at all: rows see nothing that is there
    w = s.where()
    w[2] = torch.empty((1, 0), dtype=torch.int32, device="cuda")
    out, lse = dn.dn_attn_paged(s.q.cuda(), *w)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_the_two_calls_agree_with_a_step_by_step_decode(cuda):
    """A block of 16 tokens in one call sees what 16 single-token calls see."""
    s = Setup([16], [400], 2, 128, 16, "f16", "io", group=2)
    w = s.where()
    block, _ = dn.dn_attn_paged(s.q.cuda(), *w)
    for i in range(16):
        w1 = [torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([385 + i], dtype=torch.int32, device="cuda")] + w[2:]
        one, _ = dn.dn_attn_paged(s.q[i:i + 1].cuda(), *w1)
        assert (one[0].float() - block[i].float()).abs().max() <= 2.0 ** -9 * block[i].float().abs().max()


# ---- refusals of the binding --------------------------------------------------------------------

def test_binding_refusals(cuda):
    s = Setup([3], [20], 2, 64, 16, "f16", "e4m3")
    w, q = s.where(), s.q.cuda()
    k, v = (x.cuda() for x in s.new)
    bad = lambda i, t: w[:i] + [t] + w[i + 1:]  # noqa: E731
    for wrong in (bad(0, w[0].long()), bad(0, w[0][:1]), bad(1, w[1].float()), bad(2, w[2].t()), bad(5, None), bad(5, w[5][:-1]),
                  bad(4, w[4][:-1]), bad(6, w[6].int())):
        with pytest.raises(ValueError):
            dn.dn_attn_paged(q, *wrong)
        with pytest.raises(ValueError):
            dn.dn_kv_append(k, v, *wrong)
    for q2 in (q[:, :1], q.transpose(1, 2), q.cpu(), q.to(torch.float64)):
        with pytest.raises(ValueError):
            dn.dn_attn_paged(q2, *w)
    with pytest.raises(dn.DnError):
        dn.dn_attn_paged(q.float(), *w)
    with pytest.raises(dn.DnError):
        dn.dn_attn_paged(q, *w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dn.DnError):
        dn.dn_attn_paged(q, *w, scale=-1.0)
    with pytest.raises(ValueError):
        dn.dn_attn_paged(q, *w, out=torch.empty((3, 2, 64), device="cuda"))
    with pytest.raises(ValueError):
        dn.dn_kv_append(k, v[:2], *w)
    with pytest.raises(ValueError):
        dn.dn_kv_gather(*w, k, v.bfloat16())
