"""What is measured of the paged-cache operators, and their plain forms.

Three operators of a hybrid model's attention layers, next to the recurrent state that its other
layers keep: the keys and values of new tokens written to a paged cache (``dn_kv_append``), a stretch
of the cache read back (``dn_kv_gather``), and the attention of each request's newest tokens over it
(``dn_attn_paged``). The cache holds the inputs' type, or 8 bits: e4m3 values with one power-of-two
exponent for each token and head.

``run`` computes them in elementary torch operations in 32 bits (``own`` false), or through the
library's entry points (``own`` true). ``exact`` has the definitions in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
_IO = {"f16": torch.float16, "bf16": torch.bfloat16}
# bytes per second and operations per second that a drawn case's cost is reckoned with
_HBM, _MMA = 6.8e12, 1.9e15


# ---- cases ---------------------------------------------------------------------------------


def _case(name, op, B, new, ctx, heads_kv, group, D, page, io, cache, ragged=0, window=0):
    c = dict(op=op, B=B, new=new, ctx=ctx, heads_kv=heads_kv, group=group, D=D, page=page, io=io, cache=cache,
             ragged=ragged, window=window)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's 16-token verify block written behind a 25,000-token document: the smallest call
        _case("append_verify_f16", "append", 1, 16, 25000, 4, 1, 256, 64, "f16", "io"),
        # a whole 25,000-token document written at once, rounded to 8 bits on the way
        _case("append_prompt_e4m3", "append", 1, 25000, 25000, 8, 1, 128, 64, "bf16", "e4m3"),
        # a batch of 64 requests with up to 16 accepted tokens each, small pages that end anywhere
        _case("append_batch_e4m3", "append", 64, 16, 9000, 4, 1, 64, 16, "f16", "e4m3", ragged=1),
        # a cached document's keys and values read back in full (moved to another pool, or inspected)
        _case("gather_document_e4m3", "gather", 1, 25000, 25000, 4, 1, 256, 64, "f16", "e4m3"),
        # the last few hundred tokens of several requests, for a recomputation
        _case("gather_ragged_bf16", "gather", 7, 700, 5000, 8, 1, 64, 16, "bf16", "io", ragged=2),
        # one new token of one user after a short prompt: latency
        _case("attn_one_token_f16", "attn", 1, 1, 1000, 4, 6, 256, 64, "f16", "io"),
        # one user's 16-token verify block over a 25,000-token document
        _case("attn_verify_f16", "attn", 1, 16, 25000, 4, 6, 256, 64, "f16", "io"),
        # the same block at the longest context, in 8 bits because it would not fit otherwise
        _case("attn_verify_long_e4m3", "attn", 1, 16, 268000, 4, 6, 256, 64, "bf16", "e4m3"),
        # batch mode: 64 requests of all lengths, 4-token verify blocks, 8-bit cache
        _case("attn_batch_e4m3", "attn", 64, 4, 25000, 8, 4, 128, 64, "f16", "e4m3", ragged=3),
        # 64 requests decoding one token each without drafts, small pages
        _case("attn_batch_one_bf16", "attn", 64, 1, 8000, 8, 4, 128, 16, "bf16", "io", ragged=4),
        # the last chunk of a 25,000-token prompt
        _case("attn_chunk_bf16", "attn", 1, 2048, 25000, 8, 4, 128, 64, "bf16", "io"),
        # layers that look back 1,000 tokens: prompts' chunks of odd sizes together
        _case("attn_window_e4m3", "attn", 3, 1500, 9000, 4, 8, 64, 32, "bf16", "e4m3", ragged=5, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    n, kv = lengths(c)
    pairs = c["B"] * c["heads_kv"] * c["group"] * max(n) * max(kv) if c["op"] == "attn" else 0
    held = c["B"] * max(kv) * c["heads_kv"] * c["D"]
    return max(w["bytes"] / _HBM, w["flops"] / _MMA), pairs, held


def draw(rng):
    top = [_cost(c) for c in listed()]
    top = [max(t[i] for t in top) for i in range(3)]
    while True:
        op = rng.choice(["append", "gather", "attn", "attn", "attn"])
        B = _log(rng, 1, 64)
        new = _log(rng, 1, 25000) if op != "attn" else rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 2500)])
        ctx = max(new, _log(rng, 1, 268000) if B < 4 else _log(rng, 1, 25000))
        c = _case("", op, B, new, ctx, rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 6, 7, 8]) if op == "attn" else 1,
                  rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"]), rng.choice(["io", "e4m3"]),
                  ragged=rng.randrange(1, 1000) if rng.random() < 0.6 else 0,
                  window=_log(rng, 1, 4096) if op == "attn" and rng.random() < 0.25 else 0)
        if all(a <= b for a, b in zip(_cost(c), top)):
            return c


def lengths(case):
    """New tokens and cached tokens (these included) of each request. They are the case's, whatever the seed."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    r = random.Random(case["ragged"])
    n = [new] + [r.randint(1, new) for _ in range(B - 1)]
    return n, [ctx] + [max(n[b], r.randint(max(1, ctx // 8), ctx)) for b in range(1, B)]


def work(case):
    n, kv = lengths(case)
    head = case["heads_kv"] * case["D"]
    io = head * 2  # bytes of one token's keys (or values) in the inputs' type
    held = io if case["cache"] == "io" else head + case["heads_kv"]
    total, table = sum(n), 4 * (sum(-(-x // case["page"]) for x in kv) + 2 * case["B"] + 1)
    if case["op"] != "attn":
        return {"bytes": 2 * total * (io + held) + table, "flops": 0 if case["cache"] == "io" else 4 * total * head}
    win = case["window"]
    seen = read = 0
    for a, length in zip(n, kv):
        first = length - a  # position of the request's first new token
        read += min(length, a + win - 1) if win else length
        if win:
            full = min(a, max(0, length - win + 1))  # rows from the end that see a whole window
            part = a - full
            seen += full * win + part * (first + 1) + part * (part - 1) // 2
        else:
            seen += a * (first + 1) + a * (a - 1) // 2
    q = case["group"] * io
    return {"bytes": 2 * read * held + total * (2 * q + 4 * case["group"] * case["heads_kv"]) + table,
            "flops": 4 * case["group"] * head * seen}


# ---- inputs --------------------------------------------------------------------------------


def _quantised(x):
    """e4m3 values and biased exponents of rows x [..., D]: the smallest power of two 2^e with max |x| <= 448 * 2^e."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # max |x| = m * 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    return torch.ldexp(x, -e[..., None]).to(E4M3), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n, kv = lengths(case)
    B, H, D, page, io = case["B"], case["heads_kv"], case["D"], case["page"], _IO[case["io"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)

    def rows(*shape):  # keys or values: tokens differ in size
        return (randn(*shape, D) * torch.exp(0.5 * randn(*shape, 1))).to(io)

    used = [-(-x // page) for x in kv]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(table.shape[1], device=DEV)[None, :]
    cnt = torch.tensor(used, device=DEV)[:, None]
    table[at < cnt] = order[:sum(used)]
    s = dict(case=case, page_table=table)
    s["start"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    for x in "kv":
        c = rows(pages, H, page)
        if case["cache"] == "e4m3":
            s[x + "_cache"], s[x + "_exp"] = _quantised(c)
        else:
            s[x + "_cache"], s[x + "_exp"] = c, None
        del c
        if case["op"] == "append":
            s[x] = rows(sum(n), H)
        elif case["op"] == "gather":
            s[x] = torch.empty((sum(n), H, D), dtype=io, device=DEV)
    if case["op"] == "attn":
        s["q"] = randn(sum(n), H * case["group"], D).to(io)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((sum(n), H * case["group"]), dtype=torch.float32, device=DEV)
        s["scale"] = D ** -0.5
    return s


# ---- one pass ------------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else {"append": _append, "gather": _gather, "attn": _attn}[s["case"]["op"]](s)


def _run_own(s):
    from deltanet_recurrent_state_gb300 import binding as dn
    c = s["case"]
    where = (s["start"], s["kv_len"], s["page_table"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    if c["op"] == "append":
        dn.dn_kv_append(s["k"], s["v"], *where)
        return _cache(s)
    if c["op"] == "gather":
        return dn.dn_kv_gather(*where, s["k"], s["v"])
    if "workspace" not in s:  # kept like the caches, as a serving program does
        s["workspace"] = dn.attn_workspace(s["q"], s["k_cache"], s["page_table"])
    return dn.dn_attn_paged(s["q"], *where, scale=s["scale"], window=c["window"], out=s["out"], lse=s["lse"],
                            workspace=s["workspace"])


def _cache(s):
    return {x: s[x] for x in ("k_cache", "v_cache", "k_exp", "v_exp") if s[x] is not None}


def _places(s):
    """Pool page and offset of each packed token, and its request and position."""
    c, start, kv = s["case"], s["start"].long(), s["kv_len"].long()
    i = torch.arange(sum(lengths(c)[0]), device=DEV)
    b = torch.searchsorted(start, i, right=True) - 1
    pos = kv[b] - start[b + 1] + i
    return s["page_table"][b, pos // c["page"]].long(), pos % c["page"], b, pos


def _append(s):
    page, off, _, _ = _places(s)
    for x in "kv":
        if s[x + "_exp"] is None:
            s[x + "_cache"][page, :, off] = s[x]
        else:
            val, e = _quantised(s[x])
            s[x + "_cache"].view(torch.uint8)[page, :, off] = val.view(torch.uint8)
            s[x + "_exp"][page, :, off] = e
    return _cache(s)


def _held(s, x, at):
    """What the cache stands for at an index, in 32 bits."""
    if s[x + "_exp"] is None:
        return s[x + "_cache"][at].float()
    val = s[x + "_cache"].view(torch.uint8)[at].view(E4M3).float()
    return torch.ldexp(val, s[x + "_exp"][at].int()[..., None] - 127)


def _gather(s):
    page, off, _, _ = _places(s)
    return tuple(_held(s, x, (page, slice(None), off)).to(_IO[s["case"]["io"]]) for x in "kv")


def _attn(s):
    c = s["case"]
    B, H, G, D = c["B"], c["heads_kv"], c["group"], c["D"]
    n, _ = lengths(c)
    T = max(n)
    start, kv = s["start"].long(), s["kv_len"].long()
    # queries padded to T rows a request, token-major with a head's group inside
    i = torch.arange(T, device=DEV)
    src = (start[:-1, None] + i).clamp(max=sum(n) - 1)
    q = s["q"][src].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D) * s["scale"]
    # every request's pages side by side; what lies past its length is zeroed and masked
    table = s["page_table"].long().clamp(min=0)
    pos = (kv - (start[1:] - start[:-1]))[:, None] + i                      # position of each row
    j = torch.arange(table.shape[1] * c["page"], device=DEV)
    k, v = (_held(s, x, table).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D) for x in "kv")
    live = j < kv[:, None]
    v.masked_fill_(~live[:, None, :, None], 0.0)
    see = (j <= pos[:, :, None]) & live[:, None, :]
    if c["window"]:
        see &= j > pos[:, :, None] - c["window"]
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, H, T, G, -1)
    x.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, H, T * G, -1), v).view(B, H, T, G, D) / total
    lse = (top + torch.log(total))[..., 0]
    # back to packed rows
    _, _, b, p = _places(s)
    t = p - pos[b, 0]
    return out[b, :, t].reshape(-1, H * G, D).to(s["q"].dtype), lse[b, :, t].reshape(-1, H * G)


# ---- the definitions in 64 bits --------------------------------------------------------------


def _round_e4m3(y):
    """float64 values on the e4m3 grid: 3 fraction bits, exponents from -6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_quantised(x):
    x = x.double()
    big = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 448.0))
    e = torch.where(big > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(big <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(big > 0, e, torch.full_like(e, -127.0)).clamp(-127, 127)
    return _round_e4m3(x * torch.exp2(-e)[..., None]), (e + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    n, kv = lengths(case)
    page, H, G = case["page"], case["heads_kv"], case["group"]
    table = s["page_table"].long()
    start = [sum(n[:b]) for b in range(len(n) + 1)]

    def read(x, b, lo, hi):  # [H, hi - lo, D] in 64 bits
        at = torch.arange(lo, hi, device=DEV)
        p, o = table[b, at // page], at % page
        if s[x + "_exp"] is None:
            return s[x + "_cache"][p, :, o].double().transpose(0, 1)
        val = s[x + "_cache"].view(torch.uint8)[p, :, o].view(E4M3).double()
        return (val * torch.exp2(s[x + "_exp"][p, :, o].double() - 127)[..., None]).transpose(0, 1)

    if case["op"] == "append":
        r = {}
        for x in "kv":
            r[x + "_cache"] = s[x + "_cache"].double()
            if s[x + "_exp"] is not None:
                r[x + "_exp"] = s[x + "_exp"].clone()
            new, e = (s[x].double(), None) if s[x + "_exp"] is None else _exact_quantised(s[x])
            for b in range(len(n)):
                at = torch.arange(kv[b] - n[b], kv[b], device=DEV)
                r[x + "_cache"][table[b, at // page], :, at % page] = new[start[b]:start[b + 1]]
                if e is not None:
                    r[x + "_exp"][table[b, at // page], :, at % page] = e[start[b]:start[b + 1]]
        return r
    if case["op"] == "gather":
        return tuple(torch.cat([read(x, b, kv[b] - n[b], kv[b]).transpose(0, 1) for b in range(len(n))]) for x in "kv")
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b in range(len(n)):
        first = kv[b] - n[b]
        lo = max(0, first - case["window"] + 1) if case["window"] else 0
        k, v = read("k", b, lo, kv[b]), read("v", b, lo, kv[b])
        j = torch.arange(lo, kv[b], device=DEV)[None, :]
        for h in range(H):
            for t0 in range(0, n[b], 512):
                t1 = min(n[b], t0 + 512)
                rows = slice(start[b] + t0, start[b] + t1)
                q = s["q"][rows, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,jd->tgj", q, k[h]) * s["scale"]
                pos = torch.arange(first + t0, first + t1, device=DEV)[:, None]
                hide = (j > pos) | (j <= pos - case["window"]) if case["window"] else j > pos
                x = x.masked_fill(hide[:, None, :], -math.inf)
                lse[rows, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(x, -1), v[h])
    return out, lse
