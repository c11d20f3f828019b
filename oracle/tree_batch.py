"""Trees of drafted tokens in batches: rotation of rows, attention of tree nodes by
masks, the best continuations of beams, rows moved within a cache (test
infrastructure only).  float64 throughout; the order of continuations is that of
their float64 scores.
"""
import numpy as np


def rotate(x: np.ndarray, at, freqs):
    """x [n, H, D] turned to positions at [n]: pairs (i, i + D / 2) by at * freqs[i]."""
    x = np.asarray(x, np.float64)
    half = x.shape[-1] // 2
    a = (np.asarray(at, np.float64)[:, None] * np.asarray(freqs, np.float64))[:, None]
    x1, x2 = x[..., :half], x[..., half:]
    return np.concatenate([x1 * np.cos(a) - x2 * np.sin(a), x2 * np.cos(a) + x1 * np.sin(a)], -1)


def path_masks(parents, words: int) -> np.ndarray:
    """Bits of each slot's path, itself included, int32 [slots, words]; parents[s] < s or -1."""
    out = np.zeros((len(parents), words), np.uint32)
    for s, p in enumerate(parents):
        if p >= 0:
            out[s] = out[p]
        out[s, s // 32] |= np.uint32(1 << (s % 32))
    return out.view(np.int32)


def sees(n: int, keys: int, pos: int, base: int, mask) -> np.ndarray:
    """[n, keys]: whether row i (at position pos + i) reads key t."""
    bits = (np.asarray(mask).view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1
    bits = bits.reshape(len(bits), -1).astype(bool)
    t = np.arange(keys)
    slot = t - base
    inside = (slot >= 0) & (slot < bits.shape[1])
    out = np.zeros((n, keys), bool)
    out[:, inside] = bits[:, slot[inside]]
    out[:, slot < 0] = True
    return out & (t[None] <= pos + np.arange(n)[:, None])


def masked_attention(q, k, v, see, scale):
    """q [n, Hq, D], k and v [keys, Hkv, D], see [n, keys] -> (o, mean |v|) as
    chunk_attention's; keys that a row does not read have no part in it."""
    n, hq, d = q.shape
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    o, w = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    g = hq // k.shape[1]
    for i in range(n):
        at = np.flatnonzero(see[i])
        if not len(at):
            continue
        for h in range(k.shape[1]):
            kk, vv = k[at, h], v[at, h]
            s = q[i, h * g:(h + 1) * g] @ kk.T * scale
            e = np.exp(s - s.max(-1, keepdims=True))
            e /= e.sum(-1, keepdims=True)
            o[i, h * g:(h + 1) * g], w[i, h * g:(h + 1) * g] = e @ vv, e @ np.abs(vv)
    return o, w


def beam_select(logits, score, n_best: int, temperature: float, state=None, slot: int = -1):
    """One sequence: logits [n_beams, V], score [n_beams] -> (token, parent, score float64,
    state or None, gap: the smallest difference between chosen neighbours of unlike beams)."""
    z = np.asarray(logits, np.float32).astype(np.float64)
    found = []
    for j, s in enumerate(np.asarray(score, np.float64)):
        row = np.where(np.isnan(z[j]), -np.inf, z[j])
        top = row.max()
        if not np.isfinite(s) or not np.isfinite(top):
            continue
        t = row / float(np.float32(temperature))
        lse = t.max() + np.log(np.exp(t - t.max()).sum())
        order = np.lexsort((np.arange(len(row)), -row))[:n_best + 1]
        found += [(-(s + t[v] - lse), j, -row[v], v) for v in order if row[v] > -np.inf]
    found.sort()
    gaps = [b[0] - a[0] for a, b in zip(found[:n_best], found[1:n_best + 1]) if a[1] != b[1]]
    found = found[:n_best]
    token = np.array([f[3] for f in found] + [-1] * (n_best - len(found)))
    parent = np.array([f[1] for f in found] + [-1] * (n_best - len(found)))
    out = np.array([-f[0] for f in found] + [-np.inf] * (n_best - len(found)))
    new = None
    if state is not None:
        state = np.asarray(state).view(np.uint32)
        new = np.zeros((n_best, state.shape[1]), np.uint32)
        for r, f in enumerate(found):
            new[r] = state[f[1]]
            if slot >= 0:
                new[r, (slot + r) // 32] |= np.uint32(1 << ((slot + r) % 32))
        new = new.view(np.int32)
    return token, parent, out, new, min(gaps, default=np.inf)


def moved(rows: np.ndarray, to: int, src) -> np.ndarray:
    """rows [positions, ...] with row src[i] at to + i; all read before any is written."""
    out = rows.copy()
    out[to:to + len(src)] = rows[np.asarray(src, int)]
    return out
