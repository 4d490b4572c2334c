"""Norm, rotation and attention of heads between two linears, in float64.

Written from the formulas:
  norm      y = x / sqrt(mean(x^2) + eps) * weight, per head
  rotation  the pair (a, b) as the complex number a + ib, times amplitude * e^(i angle),
            angle = 2 pi position * turns[pair]
  attention softmax(scale q k^T) v over the keys that a row sees
  cache     row s % page_size of page s // page_size holds slot s

Each function that is compared with a rounded result also returns what its error is
measured by: the sum of the magnitudes that the last sums run over.
"""

from __future__ import annotations

import numpy as np


def norm(x, weight=None, eps=1e-6):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def _pair_index(rot_dim, interleaved):
    j = np.arange(rot_dim // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot_dim // 2)


def rotate(x, positions, turns, interleaved=False, amplitude=1.0):
    """x [T, H, D]; returns (rotated, magnitude): magnitude is |a| + |b| of each pair (|x| past
    the rotated part)."""
    y = np.array(x, np.float64)
    mag = np.abs(y)
    rot = 2 * len(turns)
    if rot == 0:
        return y, mag
    around = np.outer(np.asarray(positions, np.float64), np.asarray(turns, np.float64))
    around -= np.round(around)
    z = amplitude * np.exp(2j * np.pi * around)[:, None, :]
    ia, ib = _pair_index(rot, interleaved)
    w = (y[..., ia] + 1j * y[..., ib]) * z
    both = amplitude * (mag[..., ia] + mag[..., ib])
    y[..., ia], y[..., ib] = w.real, w.imag
    mag[..., ia] = mag[..., ib] = both
    return y, mag


def attend(q, k, v, scale, seen=None):
    """Rows q [n, D] over keys k [m, D]; row i sees the first seen[i] keys (None: all).

    Returns (out [n, D], spread [n, D], reach): spread = sum p |v| / sum p, reach = the
    largest sum |q_i k_i| scale of a dot product. A row that sees no key is zero."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, m = q.shape[0], k.shape[0]
    out, spread = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    if m == 0 or n == 0:
        return out, spread, 0.0
    s = scale * (q @ k.T)
    if seen is not None:
        s = np.where(np.arange(m)[None, :] < np.asarray(seen)[:, None], s, -np.inf)
    live = np.max(s, axis=1) > -np.inf
    p = np.exp(s[live] - np.max(s[live], axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    out[live], spread[live] = p @ v, p @ np.abs(v)
    return out, spread, float(abs(scale) * np.max(np.abs(q) @ np.abs(k).T))


def prompt(q, k, v, cu_q, cu_k, scale, causal=True):
    """Packed sequences: q [Tq, H, D], k, v [Tk, Hkv, D]. Rows of no sequence are NaN."""
    out = np.full(np.shape(q), np.nan)
    spread = np.zeros(np.shape(q))
    reach = 0.0
    group = q.shape[1] // k.shape[1]
    for s in range(len(cu_q) - 1):
        a, b, c, d = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        # rows and keys end together: row i of n sees keys 0 .. m - n + i
        seen = np.maximum(0, (d - c) - (b - a) + np.arange(b - a) + 1) if causal else None
        for h in range(q.shape[1]):
            out[a:b, h], spread[a:b, h], r = attend(q[a:b, h], k[c:d, h // group], v[c:d, h // group], scale, seen)
            reach = max(reach, r)
    return out, spread, reach


def gather(cache, table_row, n):
    """The first n tokens of a sequence from a paged cache [pages, page_size, Hkv, D]."""
    page_size = cache.shape[1]
    return np.stack([cache[table_row[t // page_size], t % page_size] for t in range(n)]) if n else \
        np.zeros((0,) + cache.shape[2:])


def decode(q, k_cache, v_cache, page_table, kv_len, scale):
    """One row per sequence: q [B, H, D]."""
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    reach = 0.0
    group = q.shape[1] // k_cache.shape[2]
    for s, n in enumerate(kv_len):
        k, v = gather(k_cache, page_table[s], int(n)), gather(v_cache, page_table[s], int(n))
        for h in range(q.shape[1]):
            o, sp, r = attend(q[s, h][None], k[:, h // group], v[:, h // group], scale)
            out[s, h], spread[s, h], reach = o[0], sp[0], max(reach, r)
    return out, spread, reach


def append(cache, rows, slots):
    """The cache after token t has gone to slot slots[t] (negative: nowhere)."""
    out = np.array(cache, np.float64)
    for t, s in enumerate(slots):
        if s >= 0:
            out[s // cache.shape[1], s % cache.shape[1]] = rows[t]
    return out


# ------------------------------------------------------------------ tolerances
def norm_rope_tolerance(y, magnitude, eps_out):
    """One rounding of the result (half a step: eps_out / 2 of its value), plus the fp32
    arithmetic before it. In half steps of fp32 (2^-24), relative to |a| + |b| of a pair: the
    mean square 8 products in a lane and 5 sums across lanes (13, halved by the root), the
    division and eps (2, halved), rsqrt (2 ulp: 4), two products with 1/rms and weight (2), the
    reduced angle (one rounding of at most one half turn: pi), sine and cosine (2 ulp: 4),
    the amplitude (1), the last product and sum (2): 24.7; 32 is used."""
    return eps_out / 2 * np.abs(y) + 32 * 2.0 ** -24 * magnitude


EXP2_CUBIC = 7.5e-5   # of the prompt kernel's cubic for 2^x, fp32 evaluation included


def attention_tolerance(out, spread, reach, dim, keys, exp2=EXP2_CUBIC):
    """Relative to spread = sum p |v| / sum p: each p in fp32 off by the exponential (`exp2`: the
    prompt kernel takes some from a cubic, the decode kernel none, exp2 = 0), by its score
    (dim products and sums of magnitude at most `reach`, the scaling and the difference to the
    maximum: (dim + 4) 2^-24 reach) and by 2 ulp of the other exponentials (4 2^-24): all
    three once in p and once in the total, and `keys` fp32 additions in both sums. Then p rounded to
    bf16, off by at most 2^-8 / (1 + 2^-8) of it, and the result to bf16, off by 2^-8 of its
    value, the errors so far included: with those (1 + 2^-8) the rounding of p is 2^-8, and the
    terms in fp32 are taken (1 + 2^-8)^2 < 1 + 2^-6 times."""
    fp32 = 2 * exp2 + 2 * (dim + 4) * 2.0 ** -24 * reach + (8 + 2 * keys) * 2.0 ** -24
    return (2.0 ** -8 + (1 + 2.0 ** -6) * fp32) * spread + 2.0 ** -8 * np.abs(out)
