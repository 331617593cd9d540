"""Pins of the paged cache's oracle (CPU): e4m3 against its definition and against torch's type, the
exponent rule, placement by hand, attention against closed forms; and the cases' plain forms against it."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_e4m3_decodes_as_the_type():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.decode_e4m3(codes), want, equal_nan=True)
    assert oracle.decode_e4m3(np.uint8(0x7E)) == 448 and oracle.decode_e4m3(np.uint8(1)) == 2.0 ** -9


def test_e4m3_rounds_to_nearest_even():
    g = np.random.default_rng(1)
    y = np.concatenate([g.uniform(-448, 448, 4000), g.uniform(-2.0 ** -5, 2.0 ** -5, 4000), [0.0, -0.0, 17, 19, -17, 2.0 ** -10, 3 * 2.0 ** -10]])
    y = y.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.encode_e4m3(y), want)


@pytest.mark.parametrize("big,e", [(448.0, 0), (448.0000001, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (3.5, -7), (65504.0, 8), (2.0 ** -24, -32)])
def test_exponent_is_the_least_that_holds_the_row(big, e):
    codes, E = oracle.quantise(np.array([[0.0, -big, big / 3]]))
    assert E[0] == e + 127
    assert np.abs(oracle.values(codes, E) - [[0.0, -big, big / 3]]).max() <= big / 16


def test_a_row_of_zeros_and_a_nan():
    codes, E = oracle.quantise(np.array([[0.0, 0.0], [np.nan, 2.0]]))
    assert E[0] == 0 and (codes[0] == 0).all()
    assert codes[1, 0] == 0x7F and oracle.values(codes, E)[1, 1] == 2.0


def test_placement_by_hand():
    # one request of 3 tokens behind 3 cached ones in pages of 4: positions 3, 4, 5 -> page 7 row 3, page 2 rows 0, 1
    table = np.array([[7, 2, -1]])
    cache = np.zeros((8, 1, 4, 1))
    rows = np.array([1.0, 2.0, 3.0]).reshape(3, 1, 1)
    got = oracle.kv_append(rows, [0, 3], [6], table, cache)
    assert got[7, 0, 3, 0] == 1 and got[2, 0, 0, 0] == 2 and got[2, 0, 1, 0] == 3 and got.sum() == 6
    assert np.array_equal(oracle.kv_gather(3, [0, 3], [6], table, got), rows)
    # positions below 0 and pages that are not there are dropped, and read as zeros
    assert oracle.kv_append(rows, [0, 3], [1], table, cache).sum() == 3
    assert oracle.kv_append(rows, [0, 3], [9], table, cache).sum() == 1 + 2  # positions 6, 7; 8 has no page
    assert oracle.kv_gather(3, [0, 3], [1], table, got).reshape(3).tolist() == [0, 0, 0]


def test_attention_closed_forms():
    g = np.random.default_rng(2)
    page, D = 4, 8
    table = np.array([[1, 0]])
    k, v = g.normal(size=(2, 1, page, D)), g.normal(size=(2, 1, page, D))
    K, V = np.concatenate([k[1, 0], k[0, 0]]), np.concatenate([v[1, 0], v[0, 0]])
    # a zero query averages what it sees; one token sees itself alone through a window of 1
    out, lse, _, _ = oracle.attn_paged(np.zeros((2, 2, D)), [0, 2], [7], table, k, v, 1.0)
    assert np.allclose(out[0, 0], V[:6].mean(0)) and np.allclose(out[1, 1], V[:7].mean(0)) and np.allclose(lse[1], np.log(7))
    out, lse, _, _ = oracle.attn_paged(g.normal(size=(2, 1, D)), [0, 2], [7], table, k, v, 1.0, window=1)
    assert np.allclose(out[:, 0], V[5:7])
    # a very long query picks its best key; rows before the first token see nothing
    q = 1e4 * K[3].reshape(1, 1, D)
    best = int(np.argmax(K[:8] @ K[3]))
    assert np.allclose(oracle.attn_paged(q, [0, 1], [8], table, k, v, 1.0)[0][0, 0], V[best])
    out, lse, _, _ = oracle.attn_paged(np.ones((3, 1, D)), [0, 3], [1], table, k, v, 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], V[0])


@pytest.mark.parametrize("wrong", ["window", "causal", "scale"])
def test_the_oracle_tells_mistakes_apart(wrong):
    g = np.random.default_rng(3)
    table = np.array([[0, 1, 2]])
    k, v, q = g.normal(size=(3, 2, 4, 8)), g.normal(size=(3, 2, 4, 8)), g.normal(size=(3, 4, 8))
    right = oracle.attn_paged(q, [0, 3], [11], table, k, v, 0.5, window=5)[0]
    other = {"window": lambda: oracle.attn_paged(q, [0, 3], [11], table, k, v, 0.5, window=4),
             "causal": lambda: oracle.attn_paged(q, [0, 3], [12], table, k, v, 0.5, window=5),
             "scale": lambda: oracle.attn_paged(q, [0, 3], [11], table, k, v, 0.51, window=5)}[wrong]()[0]
    assert np.abs(right - other).max() > 1e-2


def _cases():
    spec = importlib.util.spec_from_file_location("operators_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


@pytest.mark.parametrize("cache", ["io", "e4m3"])
@pytest.mark.parametrize("op", ["append", "gather", "attn"])
def test_the_measured_plain_forms_are_the_oracle(op, cache):
    m = _cases()
    case = m._case("", op, 3, 5, 70, 2, 3 if op == "attn" else 1, 64, 16, "f16", cache, ragged=9, window=20 if op == "attn" else 0)
    s = m.prepare(case, 4)
    n = lambda t: t.double().numpy()  # noqa: E731
    start, kv, table = s["start"].numpy(), s["kv_len"].numpy(), s["page_table"].numpy()

    def held(x):
        if cache == "io":
            return n(s[x + "_cache"])
        return oracle.values(s[x + "_cache"].view(torch.uint8).numpy(), s[x + "_exp"].numpy())

    before = {x: (s[x + "_cache"].clone(), held(x)) for x in "kv"}
    got = m.run(s)
    if op == "attn":
        out, lse, _, _ = oracle.attn_paged(n(s["q"]), start, kv, table, held("k"), held("v"), s["scale"], 20)
        assert np.abs(n(got[0]) - out).max() <= 2.0 ** -10 * np.abs(out).max() and np.abs(n(got[1]) - lse).max() < 1e-5
    elif op == "gather":
        for x, y in zip("kv", got):
            assert np.array_equal(n(y), oracle.kv_gather(len(y), start, kv, table, held(x)))
    else:
        for x in "kv":
            if cache == "io":
                assert np.array_equal(n(got[x + "_cache"]), oracle.kv_append(n(s[x]), start, kv, table, before[x][1]))
            else:
                codes, E = oracle.quantise(n(s[x]))
                old = before[x][0].view(torch.uint8).numpy()
                assert np.array_equal(got[x + "_cache"].view(torch.uint8).numpy(), oracle.kv_append(codes, start, kv, table, old))
