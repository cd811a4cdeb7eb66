"""Float64 reference of attention with changed scores and of the 8-bit cache.

Plain definitions in NumPy, one head at a time: no blocking, no online softmax.
Test infrastructure only; it shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

SCALE_MIN = 2.0 ** -100


def visible(n_q: int, n_k: int, left=None, right=None, key_len=None, doc_ids=None, prefix=None):
    """[n_q, n_k] truth values: which keys a query sees (one batch entry).

    Documents are runs of equal ids; a negative id belongs to no document."""
    see = np.zeros((n_q, n_k), dtype=bool)
    run = None
    if doc_ids is not None:
        run = np.cumsum(np.concatenate(([0], np.asarray(doc_ids)[1:] != np.asarray(doc_ids)[:-1])))
    for i in range(n_q):
        for j in range(n_k):
            near = (left is None or j >= i - left) and (right is None or j <= i + right)
            ok = near or (prefix is not None and j < prefix)
            ok = ok and (key_len is None or j < key_len)
            if run is not None:
                ok = ok and run[i] == run[j] and doc_ids[i] >= 0
            see[i, j] = ok
    return see


def _probabilities(x, see):
    x = np.where(see, x, -np.inf)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - np.where(np.isinf(m), 0.0, m))
    l = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m + np.log(l), -np.inf)[..., 0]
    return p / np.where(l > 0, l, 1.0), lse


def scores(q, k, scale, softcap=0.0, slope=0.0, at=None):
    """[n_q, n_k] scores of one head and the cap's derivative; query i stands at
    position at[i] (default i)."""
    x = q @ k.T * scale
    d = np.ones_like(x)
    if softcap > 0:
        t = np.tanh(x / softcap)
        x, d = softcap * t, 1 - t * t
    at = np.arange(q.shape[0]) if at is None else at
    return x - slope * np.abs(at[:, None] - np.arange(k.shape[0])[None, :]), d


def attention(q, k, v, see, scale, softcap=0.0, slopes=None):
    """q [B, h, n_q, d], k and v [B, h_kv, n_k, d] float64, see: one [n_q, n_k] per batch entry.
    Returns O and LSE."""
    B, h, n_q, d = q.shape
    group = h // k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros((B, h, n_q))
    for b in range(B):
        for hh in range(h):
            g = hh // group
            x, _ = scores(q[b, hh], k[b, g], scale, softcap, 0.0 if slopes is None else slopes[hh])
            p, lse[b, hh] = _probabilities(x, see[b])
            o[b, hh] = p @ v[b, g]
    return o, lse


def gradients(q, k, v, dout, see, scale, softcap=0.0, slopes=None):
    """dQ, dK, dV of attention() for dout."""
    B, h, n_q, d = q.shape
    group = h // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        for hh in range(h):
            g = hh // group
            x, slope_of_cap = scores(q[b, hh], k[b, g], scale, softcap,
                                     0.0 if slopes is None else slopes[hh])
            p, _ = _probabilities(x, see[b])
            dp = dout[b, hh] @ v[b, g].T
            ds = p * (dp - (p * dp).sum(-1, keepdims=True)) * slope_of_cap * scale
            dq[b, hh] = ds @ k[b, g]
            dk[b, g] += ds.T @ q[b, hh]
            dv[b, g] += p.T @ dout[b, hh]
    return dq, dk, dv


def decode(q, k, v, lens, scale, softcap=0.0, slopes=None, window=None):
    """n_q newest queries against the first lens[b] keys of [B, h_kv, L_max, d] caches."""
    B, h, n_q, d = q.shape
    group = h // k.shape[1]
    o, lse = np.zeros(q.shape), np.full((B, h, n_q), -np.inf)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        at = n - n_q + np.arange(n_q)
        back = at[:, None] - np.arange(n)[None, :]
        see = back >= 0
        if window is not None:
            see &= back <= window
        for hh in range(h):
            g = hh // group
            x, _ = scores(q[b, hh], k[b, g, :n], scale, softcap,
                          0.0 if slopes is None else slopes[hh], at)
            p, lse[b, hh] = _probabilities(x, see)
            o[b, hh] = p @ v[b, g, :n]
    return o, lse


_E4M3 = None


def e4m3_values():
    """The 256 e4m3 numbers by code (NaN at 0x7f and 0xff)."""
    global _E4M3
    if _E4M3 is None:
        val = np.zeros(256)
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = math.nan if (e, m) == (15, 7) else (
                m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
            val[c] = -x if c & 0x80 else x
        _E4M3 = val
    return _E4M3


def nearest_e4m3(x):
    """The e4m3 number nearest to x (ties to the even code), saturating at 448."""
    pos = e4m3_values()[:0x7f]  # ascending
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, len(pos) - 1)
    lo = hi - 1
    up, down = pos[hi] - a, a - pos[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.copysign(pos[pick], x)


def append(cache, scale, new, lens, new_lens, block, int8: bool):
    """cache: code values [B, h, L, d] (float64), scale [B, h, nblk] float32, new [B, h, n, d].
    Changes cache and scale in place.  The scale, its reciprocal and the products are float32,
    as the operator is defined."""
    B, h, L, d = cache.shape
    f32 = np.float32
    top = f32(127.0 if int8 else 448.0)

    def encode(x):
        if int8:
            return np.clip(np.rint(x.astype(np.float64)), -127, 127)
        return nearest_e4m3(x.astype(np.float64))
    for b in range(B):
        start, end = int(lens[b]), min(int(lens[b]) + int(new_lens[b]), L)
        if start >= end:
            continue
        for blk in range(start // block, (end - 1) // block + 1):
            row0 = blk * block
            a, z = max(start, row0), min(end, row0 + block)
            for hh in range(h):
                x = new[b, hh, a - start:z - start].astype(f32)
                held = scale[b, hh, blk] if a > row0 else f32(0)
                s = max(held, f32(np.abs(x).max()) / top, f32(SCALE_MIN))
                inv = f32(1) / s
                cache[b, hh, a:z] = encode(x * inv)
                if s != held and a > row0:
                    cache[b, hh, row0:a] = encode(cache[b, hh, row0:a].astype(f32) * (held * inv))
                scale[b, hh, blk] = s
