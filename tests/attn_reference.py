"""Plain 64-bit forms of the paged cache and of the target pass's attention
(include/spec_attn.h), for the tests: numpy, one sequence and head at a
time."""
import numpy as np


def e4m3_table():
    """The 256 values of an e4m3 byte (1 sign, 4 exponent, 3 mantissa bits,
    bias 7; 0x7f and 0xff are NaN, no infinities)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def quantise(x):
    """x [..., D] float64 -> (e4m3 byte values [..., D], exponents [...])."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.max(np.where(fin, np.abs(x), 0.0), axis=-1)
    e = np.zeros(a.shape, np.int64)
    nz = a > 0
    m, ex = np.frexp(a[nz])
    e[nz] = np.clip(ex - 9 + (m > 0.875), -120, 120)
    y = np.where(fin, x, 0.0) * 2.0 ** -e[..., None].astype(np.float64)
    _, ye = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    grid = 2.0 ** (ye - 4.0)
    y = np.round(y / grid) * grid
    return np.where(fin, y, np.nan), e


def positions(table, page, count):
    """(page id, slot) of positions 0..count-1."""
    j = np.arange(count)
    return np.asarray(table)[j // page], j % page


def attention(q, K, V, seen, bias_far=None, slopes=None, scale=1.0, cap=0.0):
    """One sequence: q [N, Hq, D], K, V [L, Hkv, D], seen [N, L], bias_far
    [N, L] (pos_i - pos_j).  Returns out [N, Hq, D], lse [N, Hq], and two
    bounds' ingredients: spread [N, Hq, D] = sum p |v|, floor [N, Hq, D] =
    sum |v| over seen positions / sum e^(s - max s)."""
    N, Hq, D = q.shape
    G = Hq // K.shape[1]
    out, spread, floor = (np.zeros((N, Hq, D)) for _ in range(3))
    lse = np.full((N, Hq), -np.inf)
    for h in range(Hq):
        for i in range(N):
            js = np.flatnonzero(seen[i])
            if not len(js):
                continue
            k, v = K[js, h // G], V[js, h // G]
            s = scale * (k @ q[i, h])
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - slopes[h] * bias_far[i, js]
            m = s.max()
            w = np.exp(s - m)
            l = w.sum()
            lse[i, h] = m + np.log(l)
            with np.errstate(invalid="ignore"):
                out[i, h] = w @ v / l
                spread[i, h] = w @ np.abs(v) / l
                floor[i, h] = np.abs(v).sum(0) / l
    return out, lse, spread, floor
