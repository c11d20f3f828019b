"""Batched serving step: 8-bit cache rows, attention of new rows over a
sequence's keys, probabilities, verification of drafted tokens from given
random numbers (test infrastructure only).

The quantiser is stated in single IEEE fp32 operations, because they decide
integer codes; attention and probabilities are float64; the acceptance tests
and the sampled token are exact (rational and integer arithmetic).
"""
from fractions import Fraction

import numpy as np

TINY = np.float32(2.0 ** -100)


def kv8_quantise(x: np.ndarray):
    """Rows of float32 (exact bf16 values) -> (uint8 codes, float32 scales):
    scale = a / 127, code = 128 + rint(x * (127 / a)), a = max |x|."""
    x = np.asarray(x, np.float32)
    a = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    small = ~bad & (a < TINY)
    safe = np.where(bad | small, np.float32(1), a)
    scale = (safe / np.float32(127)).astype(np.float32)
    t = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint((np.where((bad | small)[..., None], 0, x) * t[..., None]).astype(np.float32))
    codes = (q + 128).astype(np.uint8)
    scale = np.where(small, np.float32(1), np.where(bad, np.float32(np.nan), scale))
    return codes, scale.astype(np.float32)


def kv8_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """float32 (code - 128) * scale, one rounding."""
    return (codes.astype(np.float32) - np.float32(128)) * np.asarray(scale, np.float32)[..., None]


def chunk_attention(q, k, v, pos: int, have=None, scale=None):
    """q [n, Hq, D] at positions pos + i, k and v [keys, Hkv, D] at positions
    0 .. keys - 1, have [keys] (False: no such key) -> (o, mean |v|) float64
    [n, Hq, D]; the second is the weights' mean of |v|, the scale of errors in
    the weights.  Rows without a key give zeros."""
    n, hq, d = q.shape
    keys, hkv = k.shape[:2]
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    scale = d ** -0.5 if scale is None else scale
    have = np.ones(keys, bool) if have is None else have
    o, w = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        see = have & (np.arange(keys) <= pos + i)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // (hq // hkv)], v[see, h // (hq // hkv)]
            s = kk @ q[i, h] * scale
            e = np.exp(s - s.max())
            o[i, h] = e @ vv / e.sum()
            w[i, h] = e @ np.abs(vv) / e.sum()
    return o, w


def probs(logits, temperature: float):
    z = np.asarray(logits, np.float64) / temperature
    m = z.max(-1, keepdims=True)
    e = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isfinite(m), m, 0.0)))
    s = e.sum(-1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def _weights(x) -> list:
    """Whole multiples of 2^-43 of float32 values clamped to [0, 1]."""
    x = np.clip(np.nan_to_num(np.asarray(x, np.float32), nan=0.0, posinf=1.0), 0.0, 1.0)
    return np.rint(x.astype(np.float64) * 2.0 ** 43).astype(np.int64)


def verify_sample(p, q, draft, u):
    """One sequence: p [n + 1, V], q [n, V] or None, draft [n], u [n + 1] ->
    (tokens [n + 1] int64, accepted)."""
    p = np.asarray(p, np.float32)
    n, v = len(draft), p.shape[1]
    a, rest = 0, None
    while a < n and 0 <= draft[a] < v:
        x = int(draft[a])
        ux, qx, px = float(u[a]), 1.0 if q is None else float(q[a][x]), float(p[a][x])
        if np.isnan([ux, qx, px]).any() or not Fraction(ux) * Fraction(qx) < Fraction(px):
            qr = np.zeros(v, np.float32) if q is None else np.asarray(q[a], np.float32)
            if q is None:
                qr[x] = 1
            rest = p[a] - qr
            break
        a += 1
    w = _weights(p[a] if rest is None else rest)
    if w.sum() == 0:
        w = _weights(p[a])
    total, new = int(w.sum()), 0
    if total:
        t = Fraction(float(min(max(u[n], 0.0), 1 - 2.0 ** -24))) * total
        run = np.cumsum(w)
        new = int(np.searchsorted(run, t.numerator // t.denominator, side="right"))
    return np.array([int(x) for x in draft[:a]] + [new] + [-1] * (n - a)), a
