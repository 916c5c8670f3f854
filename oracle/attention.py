"""fp64 definition of the attention-side operators: partial rotary positions, frequency
scaling by parts, the cache layout's values, and shared-KV attention with a window and a
sink.  Plain numpy loops over queries, independent of the product."""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(r, base=10000.0, factor=1.0, original_len=4096.0, beta_fast=32.0,
                     beta_slow=1.0):
    f = [base ** (-2.0 * j / r) for j in range(r // 2)]
    if factor == 1.0:
        return np.array(f)
    # the (fractional) pair whose wavelength fits `beta` times into the trained length
    pair = [r * math.log(original_len / (2 * math.pi * b)) / (2 * math.log(base))
            for b in (beta_fast, beta_slow)]
    lo = max(math.floor(pair[0]), 0)
    hi = max(min(math.ceil(pair[1]), r - 1), lo + 0.001)
    out = []
    for j, fj in enumerate(f):
        g = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        out.append((1 - g) * fj + g * fj / factor)
    return np.array(out)


def partial_rope(x, pos, inv_freq, r, half=False, inverse=False, magnitude=1.0):
    """x [T, H, c] -> fp64; the last r channels rotated by (+-) pos[t] * inv_freq[j]."""
    y = np.array(x, dtype=np.float64)
    if r == 0:
        return y
    c = y.shape[2]
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, : r // 2]
    cs, sn = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :] * (-1.0 if inverse else 1.0)
    ia = np.arange(r // 2) + c - r if half else np.arange(0, r, 2) + c - r
    ib = ia + (r // 2 if half else 1)
    a, b = y[:, :, ia].copy(), y[:, :, ib].copy()
    y[:, :, ia] = magnitude * (a * cs - b * sn)
    y[:, :, ib] = magnitude * (a * sn + b * cs)
    return y


def e4m3_values():
    """Value of every E4M3 byte (S.1111.111 is NaN; there are no infinities)."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (b & 0x7F) == 0x7F:
            x = math.nan
        v[b] = -x if b & 0x80 else x
    return v


_E4M3 = e4m3_values()


def cache_values(nope, rope, fp8_scale):
    """Rows of the cache layout as fp64 [rows, c] (nope uint8 bytes, rope as floats)."""
    return np.concatenate([_E4M3[np.asarray(nope)] / fp8_scale, np.asarray(rope, np.float64)], 1)


def attend(q, K, scale, sink=None):
    """One query: q [H, c], K [rows, c] (key and value) -> out [H, c], lse [H], and the
    quantities its error bounds need: abs_out = sum p |K|, top = max_s scale sum |q||K_s|."""
    H, c = q.shape
    out, mag = np.zeros((H, c)), np.zeros((H, c))
    lse = np.full(H, -math.inf)
    x = scale * (q @ K.T)
    top = np.zeros(H) if not len(K) else abs(scale) * np.max(np.abs(q) @ np.abs(K).T, axis=1)
    for h in range(H):
        terms = list(x[h]) + ([sink[h]] if sink is not None else [])
        m = max(terms, default=-math.inf)
        if m == -math.inf:
            continue
        total = math.fsum(math.exp(v - m) for v in terms)
        lse[h] = m + math.log(total)
        p = np.exp(x[h] - lse[h])
        out[h] = p @ K
        mag[h] = p @ np.abs(K)
    return out, lse, mag, top
