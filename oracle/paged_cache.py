"""The paged cache of the attention layers: write, read back, attend. Plain NumPy, float64.

Definitions:

* position p of request b is row p % page of pool page table[b][p // page]; the request's newest
  n = start[b+1] - start[b] tokens are packed rows start[b].. and hold positions kv_len[b] - n ..;
* an 8-bit row of values x is (y, E): e = E - 127 the least integer with max |x| <= 448 * 2^e (clamped to
  -127 .. 127; a row of zeros has E = 0) and y the e4m3 value nearest to x * 2^-e, ties to the even code;
* attention of packed row t at position p over the positions j with 0 <= j <= p, j < kv_len and, with a
  window, j > p - window: out = sum_j softmax(scale q . k_j) v_j, lse the log of the sum of exponentials.

e4m3 (4 exponent bits of bias 7, 3 fraction bits, no infinity, 0x7f NaN) is decoded from its definition and
rounded to by searching its table.
"""

import numpy as np


def _decode_table():
    t = np.empty(128)
    for code in range(128):
        e, m = code >> 3, code & 7
        t[code] = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
    t[127] = np.nan
    return t


E4M3 = _decode_table()


def decode_e4m3(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    return np.where(codes & 0x80, -1.0, 1.0) * E4M3[codes & 0x7F]


def encode_e4m3(y):
    """Codes of the e4m3 values nearest to y (|y| <= 464 finite), ties to the even code; NaN to 0x7f."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.abs(np.where(np.isnan(y), 0.0, y))
    hi = np.clip(np.searchsorted(E4M3[:127], mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - E4M3[lo], E4M3[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)
    code = np.where(np.signbit(y), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(y), 0x7F, code).astype(np.uint8)


def quantise(x):
    """(codes, exponent bytes) of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    big = np.max(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    E = np.zeros(big.shape, dtype=np.uint8)
    for e in range(-127, 127):  # one more for every power of two that does not hold the row
        E += big > 448.0 * 2.0 ** e
    return encode_e4m3(np.clip(x * 2.0 ** (127.0 - E[..., None]), -448, 448)), E


def values(codes, E):
    return decode_e4m3(codes) * 2.0 ** (E[..., None].astype(np.float64) - 127)


def _place(table, b, pos, page, pages):
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    g = int(table[b, pos // page])
    return (g, pos % page) if 0 <= g < pages else None


def packed(start, kv_len, total):
    """(row, request, position) of every packed row that belongs to a request."""
    for b in range(len(kv_len)):
        n = int(start[b + 1] - start[b])
        for i in range(n):
            yield int(start[b]) + i, b, int(kv_len[b]) - n + i


def kv_append(rows, start, kv_len, table, cache):
    """cache [pages, heads, page, ...] with the rows [total, heads, ...] written to their places."""
    cache = cache.copy()
    for t, b, pos in packed(start, kv_len, len(rows)):
        at = _place(table, b, pos, cache.shape[2], cache.shape[0])
        if at is not None:
            cache[at[0], :, at[1]] = rows[t]
    return cache


def kv_gather(total, start, kv_len, table, cache):
    """rows [total, heads, D] of a cache of values [pages, heads, page, D]; zeros where there is none."""
    rows = np.zeros((total,) + cache.shape[1:2] + cache.shape[3:])
    for t, b, pos in packed(start, kv_len, total):
        at = _place(table, b, pos, cache.shape[2], cache.shape[0])
        if at is not None:
            rows[t] = cache[at[0], :, at[1]]
    return rows


def attn_paged(q, start, kv_len, table, k, v, scale, window=0):
    """out [total, heads, D], lse [total, heads], and what the error bounds of a test need: the
    probability-weighted |v| of every output, and the largest scale * sum |q| |k| of every row."""
    total, heads, D = q.shape
    pages, hk, page, _ = k.shape
    G = heads // hk
    out, lse = np.zeros(q.shape), np.full((total, heads), -np.inf)
    weight, size = np.zeros(q.shape), np.zeros((total, heads))
    for b in range(len(kv_len)):
        length = max(0, min(int(kv_len[b]), table.shape[1] * page))
        K, V = np.zeros((length, hk, D)), np.zeros((length, hk, D))
        for j in range(length):
            at = _place(table, b, j, page, pages)
            if at is not None:
                K[j], V[j] = k[at[0], :, at[1]], v[at[0], :, at[1]]
        n = int(start[b + 1] - start[b])
        for i in range(n):
            p = int(kv_len[b]) - n + i
            lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, length)
            if hi <= lo:
                continue
            t = int(start[b]) + i
            for h in range(heads):
                x = scale * (K[lo:hi, h // G] @ q[t, h])
                m = x.max()
                e = np.exp(x - m)
                out[t, h] = e @ V[lo:hi, h // G] / e.sum()
                weight[t, h] = e @ np.abs(V[lo:hi, h // G]) / e.sum()
                lse[t, h] = m + np.log(e.sum())
                size[t, h] = (scale * (np.abs(K[lo:hi, h // G]) @ np.abs(q[t, h]))).max()
    return out, lse, weight, size
