"""Plain 64-bit forms of the rotary positions, the latent attention and the log
probabilities (include/spec_attn.h, include/spec_verify.h), for the tests: numpy."""
import math

import numpy as np


def frequencies(rot, base, scaling="plain", factor=1.0, original=0, low=0.0, high=0.0):
    """theta_i in 64 bits."""
    out = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        if scaling == "linear":
            t /= factor
        elif scaling == "turns":
            w = min(1.0, max(0.0, (original * t / (2 * math.pi) - low) / (high - low)))
            t *= w + (1 - w) / factor
        elif scaling == "index":
            def at(n):
                return rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
            w = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
            t *= w + (1 - w) / factor
        out.append(t)
    return np.array(out)


def turned(x, pos, freqs, first, interleaved, amplitude=1.0, inverse=False):
    """x [..., H, D] at positions pos [...]; freqs: the 64-bit fixed point integers.
    Returns the result and, per element, |u| + |v| of its pair (0 where it stays)."""
    x = np.asarray(x, np.float64)
    half = len(freqs)
    turns = np.array([[(int(f) * int(p) % 2 ** 64) / 2.0 ** 64 for f in freqs] for p in np.ravel(pos)])
    a = 2 * math.pi * turns.reshape(*np.shape(pos), 1, half) * (-1 if inverse else 1)
    out, size = x.copy(), np.zeros_like(x)
    part = x[..., first:first + 2 * half]
    u, v = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    new = (amplitude * (u * np.cos(a) - v * np.sin(a)), amplitude * (v * np.cos(a) + u * np.sin(a)))
    for k, y in enumerate(new):
        at = slice(first + k, first + 2 * half, 2) if interleaved else slice(first + k * half, first + (k + 1) * half)
        out[..., at] = y
        size[..., at] = abs(amplitude) * (np.abs(u) + np.abs(v))
    return out, size


# How far a turned element may be off, in fp32, as a share of |u| + |v|: sine and
# cosine to 2^-23, the angle's own 2^-25, the amplitude's product and the two of
# the turn with its sum, 2^-24 each.
TURN = 2.0 ** -23 + 2.0 ** -25 + 4 * 2.0 ** -24


def latent(q, K, C, seen, scale):
    """One sequence: q [N, H, W], K [L, W], seen [N, L].  Returns out [N, H, C], lse
    [N, H], spread [N, H, C] = sum p |c|, and size [N, H] = the largest
    scale * sum |q| |k| of a seen position."""
    N, H, W = q.shape
    out, spread = np.zeros((N, H, C)), np.zeros((N, H, C))
    lse, size = np.full((N, H), -np.inf), np.zeros((N, H))
    for i in range(N):
        js = np.flatnonzero(seen[i])
        if not len(js):
            continue
        k = K[js]
        for h in range(H):
            with np.errstate(invalid="ignore"):
                s = scale * (k @ q[i, h])
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                lse[i, h] = m + np.log(total)
                out[i, h] = w @ k[:, :C] / total
                spread[i, h] = w @ np.abs(k[:, :C]) / total
                size[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, spread, size


def logprobs(x, token, T, top):
    """One row x [V]: (ln p(token), entropy, rank, ids, their ln p, largest |ln p|
    that counts: over tokens of p > e^-100)."""
    x = np.asarray(x, np.float64)
    y = x / T
    y = y - y.max()
    lz = np.log(np.exp(y).sum())
    lp = y - lz
    p = np.exp(lp)
    order = np.lexsort((np.arange(len(x)), -x))
    rank = int(np.flatnonzero(order == token)[0])
    some = p > 0
    return lp[token], -(p[some] * lp[some]).sum(), rank, order[:top], lp[order[:top]]
