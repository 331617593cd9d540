"""dn_accept_sampled where sums over a row decide: rows of a few distinct values, whose 64-bit sums are products and so known to 10^-15,
and random numbers a few 10^-11 beside a border of the running sum.

A weight is right to 2^-33 of itself. A share of a sum changes by its two sides' product, at most 1/4, times the difference of
their errors, at most 2^-32: 2^-34. Sums are taken in units of 2^-43 of the largest weight, with half a unit for each of 128
warps, twice: 2^-36. So a random number lies within the interval of its token, widened by 2^-34 + 2^-36 on either side (`TOL`, 7.3e-11).
"""

import numpy as np
import pytest
import torch

from deltanet_recurrent_state_gb300 import binding as dn

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TOL = 2.0 ** -34 + 2.0 ** -36


def value(x, dt):
    """x as the type holds it."""
    return float(torch.tensor(x, dtype=torch.float64).to(DT[dt]))


def weight(x, top, temperature):
    return np.exp((np.float64(x) - top) / np.float64(np.float32(temperature)))


def draw(logits, u, temperature, top_k=0, top_p=1.0, min_p=0.0, workspace=None):
    """Targets of rows [B, V]; the parameters are a row's each, or all rows'."""
    B = logits.shape[0]

    def column(v, dtype):
        return torch.as_tensor(np.broadcast_to(np.asarray(v), (B,)).copy()).to(dtype).cuda()

    got = dn.dn_accept_sampled(logits[:, None].cuda(), torch.zeros((B, 1), dtype=torch.int32, device="cuda"), column(u, torch.float32)[:, None],
                               column(temperature, torch.float32), column(top_k, torch.int32), column(top_p, torch.float32),
                               column(min_p, torch.float32), workspace=workspace)
    return got[0][:, 0].cpu().numpy()


# ---- a top_p whose border lies beside the least value that min_p keeps, and one between two values ----


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("B", [12, 100])
def test_top_p_reaches_the_least_value_that_min_p_keeps(cuda, B, dt):
    """Many tokens at the least kept value, below zero, a floor that is no value of the type, and a top_p that keeps all that min_p does."""
    V = 24000
    g = torch.Generator().manual_seed(B)
    logits = torch.empty((B, V), dtype=DT[dt])
    min_p = []
    for b in range(B):
        top = value(-0.25 - 0.5 * b / B, dt)
        least = value(top - 1.0, dt)
        logits[b] = (top - 1.0 * torch.rand(V, generator=g, dtype=torch.float64) ** 2).clamp(least, top).to(DT[dt])
        logits[b, torch.randint(0, V, (6000,), generator=g)] = least
        logits[b, torch.randint(0, V, (6000,), generator=g)] = least - 1.0  # (min_p leaves these out)
        logits[b, b] = top
        min_p.append(float(np.float32(weight(least, top, 1.0) * (1 - 1e-4))))
    u = (np.arange(B) + 0.5) / B
    for top_p in (1 - 2.0 ** -24, 1 - 2.0 ** -23):
        ws = dn.sample_workspace(B, 1, V, cuda)
        token = draw(logits, u, 1.0, 0, top_p, min_p, workspace=ws)
        assert int(ws.count_nonzero()) == 0
        for b in range(B):
            x = logits[b].double().numpy()
            w = np.exp(x - x.max())
            w[w < min_p[b]] = 0.0
            assert w[w > 0].min() > 4 * 2.0 ** -23 * w.sum()  # (the last token is more than what top_p leaves out)
            upto = np.cumsum(w) / w.sum()
            i = int(token[b])
            assert w[i] > 0 and upto[i] - w[i] / w.sum() - TOL <= float(np.float32(u[b])) <= upto[i] + TOL, (top_p, b, i)


@pytest.mark.parametrize("dt", list(DT))
def test_top_p_between_two_values(cuda, dt):
    """The mass down to a value is top_p's to a few 10^-10, closer than sums of the value's tokens in 32 bits come to their number times one of them."""
    top, n2 = value(9.0, dt), 3000
    one, two = value(top - 10.0, dt), value(top - 10.5, dt)
    w, w2 = weight(one, top, 1.0), weight(two, top, 1.0)
    cases = []
    for n in range(4000, 9000):
        share = (1 + n * w) / (1 + n * w + n2 * w2)
        p = np.float32(share)
        for q in (p, np.nextafter(p, np.float32(0)), np.nextafter(p, np.float32(1))):
            if 1e-10 < abs(float(q) - share) < 2e-9:
                cases.append((n, float(q), share))
    assert len(cases) >= 40
    cases = cases[:: max(1, len(cases) // 120)][:120]
    V = 12100
    logits = torch.full((len(cases), V), -float("inf"), dtype=DT[dt])
    u = np.float32(1 - 2.0 ** -24)
    for b, (n, _, _) in enumerate(cases):
        logits[b, :n2] = two
        logits[b, n2:n2 + n] = one
        logits[b, n2 + n] = top
    # the peak is the last: its border tells what is kept before it
    token = draw(logits, [0.0 if b % 2 else u for b in range(len(cases))], 1.0, 0, [c[1] for c in cases])
    for b, (n, p, share) in enumerate(cases):
        if b % 2:  # u = 0: the first kept token
            assert token[b] == (0 if p > share else n2), (b, n, p - share)
        else:
            assert token[b] == n2 + n, b


# ---- light tokens that make up much of the row, and many equal ones far below the largest ----


def beside_borders(borders, count, least=1.25 * TOL, most=5e-10):
    """Random numbers, as 32-bit floats hold them, that lie beside a border and further than TOL from it."""
    near = (borders[:, None] + np.array([-2.6, -1.6, -1.1, 1.1, 1.6, 2.6]) * 1e-10).astype(np.float32).astype(np.float64)
    off = np.abs(near - borders[:, None])
    out = np.unique(near[(off > least) & (off < most) & (near > 0) & (near < 1)])
    return out[:: max(1, len(out) // count)][:count]


def equal_light_rows(dt, top, low, temperature, n, peak_at, count):
    """The borders of a row with a peak at place peak_at among n equal tokens, and random numbers beside them."""
    w = weight(low, top, temperature)
    upto = np.arange(1, n + 2) * w + np.where(np.arange(n + 1) >= peak_at, 1 - w, 0.0)  # mass of tokens 0 .. i
    borders = upto / upto[-1]
    return borders, beside_borders(borders[:-1], count)


def check_equal_light(cuda, dt, V, top, low, temperature, n, peak_at, rows):
    borders, chosen = equal_light_rows(dt, top, low, temperature, n, peak_at, rows)
    assert len(chosen) >= min(rows, 20), len(chosen)
    row = torch.full((V,), -float("inf"), dtype=DT[dt])
    row[: n + 1] = low
    row[peak_at] = top
    u = chosen
    want = np.searchsorted(borders, u, side="right")  # the first token whose border is above u
    for batch in (len(u), 6):  # rows that fill the GPU, and a few
        token = draw(row[None].expand(batch, V).contiguous(), u[:batch], temperature)
        bad = token != want[:batch]
        assert not bad.any(), (temperature, n, peak_at, bad.sum(), token[bad][:5], want[:batch][bad][:5])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("share", [0.3, 0.02])
@pytest.mark.parametrize("temperature", [1.0, 1.37])
def test_many_equal_tokens_beside_a_peak(cuda, temperature, share, dt):
    """Equal tokens lose as much, each, in a sum of 32 bits."""
    V, top = 151936, 6.0
    for n, peak_at in ((150000, 150000), (131000, 70000), (90001, 45000)):
        low = value(top + temperature * np.log(share / n), dt)
        check_equal_light(cuda, dt, V, top, low, temperature, n, peak_at, 100)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("far", [37.3, 39.4, 40.6, 42.2, 44.5])
def test_ties_far_below_the_largest(cuda, far, dt):
    """top_k cuts through equal tokens of less than a unit of the sums: 10,000 and more of them, and their mass is counted to less than a unit each."""
    V = 120000
    top = 20.0
    low = value(top - far * np.log(2.0), dt)
    w = weight(low, top, 1.0)
    for B in (4, 100):
        top_k = [1 + (110000, 40000, 10001, 2000)[b % 4] for b in range(B)]
        logits = torch.full((B, V), low, dtype=DT[dt])
        logits[:, -1] = top
        light = np.array([(k - 1) * w for k in top_k])
        border = light / (1 + light)  # where the peak begins
        for off in (2 * TOL, -2 * TOL):
            u = np.float32(border + off)
            token = draw(logits, u, 1.0, top_k)
            for b in range(B):
                if float(u[b]) >= border[b] + TOL:
                    assert token[b] == V - 1, (top_k[b], token[b])
                elif 0 < float(u[b]) <= border[b] - TOL:  # the token whose interval holds u, or one within TOL
                    total = 1 + light[b]
                    assert abs(float(u[b]) * total - token[b] * w) <= TOL + w and token[b] < top_k[b] - 1, (top_k[b], token[b])


# ---- light tokens: a peak, and many tokens of less than 2^-14 of its weight ----


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("temperature", [1.0, 1.1, 1.3, 0.7])
def test_a_share_of_light_tokens_below_the_limit(cuda, temperature, dt):
    """Equal tokens that make up nearly 2^-10 of the row: their 32-bit sums have errors of one sign."""
    V, top = 151936, 4.0
    n = 150000
    low = value(top + temperature * np.log(0.9 * 2.0 ** -10 / n), dt)
    n = min(n, int(0.95 * 2.0 ** -10 / weight(low, top, temperature)))
    check_equal_light(cuda, dt, V, top, low, temperature, n, n, 160)


@pytest.mark.parametrize("dt", list(DT))
def test_unequal_light_tokens_below_the_limit(cuda, dt):
    """The same with a normal distribution of them, and a peak at the end."""
    V = 151936
    x = (2 * torch.randn(V, generator=torch.Generator().manual_seed(3), dtype=torch.float64)).to(DT[dt])
    for temperature in (1.1, 1.3, 0.9):
        rest = x[:-1].double().numpy()
        t64 = float(np.float32(temperature))
        x[-1] = float(t64 * np.log(np.exp(rest / t64).sum() / (0.9 * 2.0 ** -10)))
        w = np.exp((x.double().numpy() - float(x[-1])) / t64)
        part = w[:151900].reshape(-1, 100)  # (sums of 100, so that 64 bits are enough)
        upto = np.concatenate([[0], np.cumsum(part.sum(1))[:-1]])[:, None] + np.cumsum(part, 1)
        borders = upto.ravel() / (part.sum() + w[151900:].sum())
        u = beside_borders(borders[50000:], 160)
        want = np.searchsorted(borders, u, side="right")
        token = draw(x[None].expand(len(u), V).contiguous(), u, temperature)
        assert len(u) >= 100 and (token == want).all(), (temperature, (token != want).sum())


@pytest.mark.parametrize("dt", list(DT))
def test_top_p_among_light_tokens(cuda, dt):
    """A share of light tokens below the limit, and a top_p whose border lies a few 10^-10 beside one of theirs."""
    V, top, temperature = 40000, 4.0, 1.1
    low = value(top + temperature * np.log(0.9 * 2.0 ** -10 / 39000), dt)
    w = weight(low, top, temperature)
    most = min(39000, int(0.98 * 2.0 ** -10 / w))
    cases = []
    for n in range(most - 6000, most):
        for step in range(1, 400):
            p = 1 - step * 2.0 ** -24
            kept = (p * (1 + n * w) - 1) / w  # of the light tokens
            off = (kept - np.rint(kept)) * w
            if 1 < kept < n - 1 and 1.25 * TOL < abs(off) < 5e-10:
                cases.append((n, p, int(np.ceil(kept))))
    assert len(cases) >= 200
    cases = cases[:: len(cases) // 160][:160]
    logits = torch.full((len(cases), V), -float("inf"), dtype=DT[dt])
    u = float(np.float32(1 - 2.0 ** -24))
    for b, (n, _, _) in enumerate(cases):
        logits[b, 0] = top
        logits[b, 1:n + 1] = low
    token = draw(logits, u, temperature, 0, [c[1] for c in cases])
    for b, (n, p, kept) in enumerate(cases):
        total = 1 + kept * w
        # the last kept token, or one before it: total * 2^-24 from the end; a border that is as near as TOL leaves two
        want = {int(np.floor((float(u) * total + s * TOL - 1) / w)) + 1 for s in (-1, 1)}
        assert int(token[b]) in want, (n, p, kept, token[b], want)


# ---- histograms of masses: more tokens of a CTA in one bin than 32 bits hold as 16-bit shares ----


@pytest.mark.parametrize("B,V", [(40, 151936), (60, 151936), (20, 400000)])
def test_nearly_constant_rows_of_a_few_ctas(cuda, B, V):
    """Right, and in few passes: a row costs no more than six times one of the same values that has eight CTAs."""
    g = torch.Generator().manual_seed(B)
    logits = torch.randn((B, V), generator=g)
    u = torch.rand(B, generator=g).numpy()
    token = draw(logits, u, 1000.0, 0, 0.95)
    for b in range(0, B, 9):
        x = logits[b].double().numpy()
        w = np.exp((x - x.max()) / 1000.0)
        order = np.argsort(-x, kind="stable")
        upto = np.cumsum(w[order])
        kept = np.sort(order[: int(np.searchsorted(upto, float(np.float32(0.95)) * upto[-1])) + 1])
        upto = np.cumsum(w[kept]) / w[kept].sum()
        i = int(np.searchsorted(kept, token[b]))
        assert i < len(kept) and kept[i] == token[b]
        # (64-bit sums of 150,000 are right to 10^-11)
        assert (upto[i - 1] if i else 0.0) - TOL - 1e-11 <= u[b] <= upto[i] + TOL + 1e-11

    def timed(rows):
        args = [logits[:rows, None].cuda(), torch.zeros((rows, 1), dtype=torch.int32, device="cuda"), torch.tensor(u[:rows, None]).cuda(),
                torch.full((rows,), 1000.0, device="cuda"), None, torch.full((rows,), 0.95, device="cuda")]
        ws = dn.sample_workspace(rows, 1, V, cuda)
        times = []
        for _ in range(6):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(5):
                dn.dn_accept_sampled(*args, workspace=ws)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        return min(times)

    few = timed(9)  # eight CTAs a row, below the limit
    assert timed(B) < 6 * (8 / (4 if V == 400000 else 2)) * few


# ---- one weight at a time ----


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("V", [1800, 20000])
def test_weights_of_many_sizes(cuda, V, dt):
    """Equal tokens before a peak, other ones in every row, a few octaves below it: their one weight decides where the peak begins, and a random number lies
    beside that place."""
    rng = np.random.default_rng(V)
    N = 400000
    temperature = np.exp(rng.uniform(-1, 1, N)).astype(np.float32)
    low = torch.tensor(3.0 - temperature * rng.uniform(0.05, 7.0, N)).to(DT[dt]).double().numpy()
    w = np.exp((low - 3.0) / temperature.astype(np.float64))
    n = np.clip(np.rint(rng.uniform(0.4, 0.9, N) / w), 1, 1700).astype(np.int64)
    border = n * w / (1 + n * w)
    u = border.astype(np.float32)
    off = u - border
    chosen = np.flatnonzero((np.abs(off) > 1.25 * TOL) & (np.abs(off) < 1.6e-10))[:400]
    assert len(chosen) >= 300
    logits = torch.full((len(chosen), V), -float("inf"), dtype=DT[dt])
    for b, i in enumerate(chosen):
        logits[b, : n[i]] = float(low[i])
        logits[b, n[i]] = 3.0
    want = np.where(off[chosen] < 0, n[chosen] - 1, n[chosen])
    for top_k in (0, V, 1701):
        token = draw(logits, u[chosen], temperature[chosen], top_k)
        assert (token == want).all(), (token != want).sum()
    for b in range(0, len(chosen), 20):  # a row alone
        assert draw(logits[b:b + 1], u[chosen[b]], temperature[chosen[b]])[0] == want[b]


# ---- the last kept token ----


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("B,V", [(4, 600), (4, 40000), (100, 40000)])
def test_random_numbers_of_one_and_more(cuda, B, V, dt):
    """They give the last kept token, and may leave out one of less than 2^-41 of the largest weight."""
    top = 20.0
    last = [40.5, 60.0, 42.5]  # a row's last token's weight, in octaves below the largest
    logits = torch.full((B, V), value(top - 12.0, dt), dtype=DT[dt])
    logits[:, 5] = top
    for i in range(3):
        logits[i::3, -1] = value(top - last[i] * np.log(2.0), dt)
    light = np.arange(B) % 3 != 0
    for u in (1.0, 2.0, float("inf")):
        for top_k in (0, V):
            token = draw(logits, u, 1.0, top_k)
            assert ((token == V - 1) | (light & (token == V - 2))).all()
    logits[:, 10:-1] = -float("inf")  # few tokens are left: they are listed, in finer units
    for top_k in (V, 200):
        token = draw(logits, 1.0, 1.0, top_k)
        assert ((token == V - 1) | (light & (token == 9))).all()
