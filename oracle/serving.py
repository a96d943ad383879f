"""The serving step over a KV cache in 8 bits: plain numpy fp64 definitions.

TEST INFRASTRUCTURE ONLY: the tests and ``__graft_entry__.smoke()`` are its
users.  The CUDA library never imports or calls it; the two share no code.

  rope         pair (a, b) of a row at position p turns by p f_i
  quantise     e4m3 codes with one power-of-two scale per group and head
  append_q8    rows written behind a prefix, their groups requantised
  decode       masked softmax attention over codes times scales
  verify       speculative sampling from given random numbers

Whole numbers and codes are exact; the rest is fp64.
"""
from __future__ import annotations

import numpy as np


# ----------------------------------------------------------------------------
# rotary positions


def rope(x, pos, inv_freq, interleaved=False, mscale=1.0, adjoint=False):
    """x [B, H, N, d] float64, pos [B, N] integers, inv_freq [rot / 2]."""
    x = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = len(f)
    y = x.copy()
    t = np.asarray(pos)[:, None, :].astype(np.float64)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(t * f[i]), np.sin(t * f[i])
        if adjoint:
            s = -s
        y[..., a] = mscale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = mscale * (x[..., b] * c + x[..., a] * s)
    return y


def rope_freqs(rot, base, scaling="plain", factor=1.0, trained_len=0, fast=32.0, slow=1.0):
    out = []
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            w = (trained_len * f / (2 * np.pi) - slow) / (fast - slow)
            w = min(1.0, max(0.0, w))
            f = (1 - w) * f / factor + w * f
        out.append(f)
    m = 0.1 * np.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return np.array(out), m


# ----------------------------------------------------------------------------
# e4m3


def e4m3_table() -> np.ndarray:
    """The 256 values of 1 + 4 + 3 bits, bias 7; 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -v if c & 128 else v
    return out


_TABLE = e4m3_table()
_POSITIVE = _TABLE[:127]  # increasing: 0 .. 448


def e4m3_encode(x, top=448.0) -> np.ndarray:
    """Nearest code, ties to the even code, +-top (a code) beyond it."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), top)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    down, up = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(127), code)


def e4m3_decode(codes) -> np.ndarray:
    return _TABLE[np.asarray(codes, dtype=np.uint8)]


def group_scale(values) -> float:
    """The smallest power of two, 2^-64 or more, with |x| <= 448 s for the
    finite values."""
    v = np.abs(np.asarray(values, dtype=np.float64)).ravel()
    v = v[np.isfinite(v)]
    top = v.max() if v.size else 0.0
    k = -64
    while top > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append_q8(codes, scale, cache_len, new, n_new, group):
    """codes uint8 [B, H, S, d], scale [B, H, groups], new [B, H, b, d] float64.
    Returns the codes and scales afterwards.  At the scale 2^120 codes are at
    most 240: the next one stands for 2^128, beyond fp32 and bf16."""
    codes, scale = codes.copy(), np.array(scale, dtype=np.float64)
    B, H, S, d = codes.shape
    for i in range(B):
        a, n = int(cache_len[i]), int(n_new[i])
        if a < 0 or n < 0 or n > new.shape[2] or a + n > S:
            continue
        for h in range(H):
            for g in range(a // group, (a + n + group - 1) // group if n else 0):
                p0, p1 = g * group, min((g + 1) * group, a + n)
                rows = [e4m3_decode(codes[i, h, p]) * scale[i, h, g] if p < a else new[i, h, p - a]
                        for p in range(p0, p1)]
                s = group_scale(rows)
                for p, r in zip(range(p0, p1), rows):
                    codes[i, h, p] = e4m3_encode(r / s, 240.0 if s == 2.0 ** 120 else 448.0)
                scale[i, h, g] = s
    return codes, scale


def values(codes, scale, group):
    S = codes.shape[2]
    return e4m3_decode(codes) * np.repeat(np.asarray(scale, dtype=np.float64), group, axis=2)[:, :, :S, None]


# ----------------------------------------------------------------------------
# attention


def decode(q, k, v, cache_len, mode):
    """q [B, Hq, b, d], k, v [B, Hkv, S, d] float64.  Returns out, lse, and
    for error bounds mag = sum_j p_j |v_j| and qk = max_j sum_e |q_e k_je|."""
    B, Hq, b, d = q.shape
    H = k.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, Hq, b), -np.inf)
    mag, qk = np.zeros(q.shape), np.zeros((B, Hq, b))
    for i in range(B):
        for h in range(Hq):
            g = h // (Hq // H)
            for j in range(b):
                n = int(cache_len[i]) + (b, j + 1, 0)[mode]
                if n == 0:
                    continue
                kk, vv = k[i, g, :n], v[i, g, :n]
                x = kk @ q[i, h, j] / np.sqrt(d)
                m = x.max()
                e = np.exp(x - m)
                p = e / e.sum()
                out[i, h, j], lse[i, h, j] = p @ vv, m + np.log(e.sum())
                mag[i, h, j], qk[i, h, j] = p @ np.abs(vv), (np.abs(kk) @ np.abs(q[i, h, j])).max()
    return out, lse, mag, qk


# ----------------------------------------------------------------------------
# verification


def draw_from(weights, r: float) -> int:
    w = np.where(np.isnan(weights), 0.0, np.maximum(weights, 0.0))
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    over = np.nonzero((c > r * c[-1]) & (w > 0))[0]
    return int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])


def verify_one(draft, q, p, u, r):
    """draft [n], q [n, V] or None, p [n + 1, V], u [n], r.  (accepted, next)."""
    n = len(draft)
    for j, x in enumerate(draft):
        qj = float(q[j][x]) if q is not None else 1.0
        if not float(u[j]) * qj < float(p[j][x]):
            pj = np.asarray(p[j], dtype=np.float64)
            if q is not None:
                rest = pj - np.asarray(q[j], dtype=np.float64)
            else:
                rest = pj.copy()
                rest[x] -= 1.0
            t = draw_from(rest, float(r))
            return j, t if t >= 0 else draw_from(pj, float(r))
    return n, draw_from(np.asarray(p[n], dtype=np.float64), float(r))
