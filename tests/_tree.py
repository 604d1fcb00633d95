"""Attention of a drafted tree over the 4-bit cache in 64 bits on the CPU, from its definition."""
import numpy as np


def sees(words, T, n):
    """(T, n) booleans: draft i sees key j of a sequence of n keys."""
    j = np.arange(n)[None]
    bit = j - (n - T)
    w = np.array([int(x) & (2 ** 64 - 1) for x in words], dtype=np.uint64)[:, None]
    named = (w >> np.clip(bit, 0, 63).astype(np.uint64)) & np.uint64(1)
    return (bit < 0) | ((bit < T) & (named == 1))


def attention(q, words, ks, vs, scale):
    """o, lse, sum p |v| and the largest scale * sum |q k| of a row (see _qcache.attention)."""
    q = q.double().cpu().numpy()
    B, H, T, d = q.shape
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full((B, H, T), -np.inf), np.zeros((B, H, T))
    for b in range(B):
        Hkv, n, _ = ks[b].shape
        if n == 0:
            continue
        seen = sees(words[b].tolist(), T, n)
        any_key = seen.any(-1)
        for h in range(H):
            k, v = ks[b][h * Hkv // H], vs[b][h * Hkv // H]
            s = np.where(seen, scale * (q[b, h] @ k.T), -np.inf)
            top = np.where(any_key, s.max(-1), 0.0)[:, None]
            e = np.exp(s - top)
            total = e.sum(-1)
            with np.errstate(divide="ignore"):
                lse[b, h] = top[:, 0] + np.log(total)
            p = e / np.where(total > 0, total, 1.0)[:, None]
            o[b, h], mag[b, h] = p @ v, p @ np.abs(v)
            big[b, h] = np.where(any_key, scale * np.where(seen, np.abs(q[b, h]) @ np.abs(k).T, 0.0).max(-1), 0.0)
    return o, lse, mag, big


def random_parents(B, T, rng):
    """Parents before children; -1: a child of the last accepted token."""
    p = np.stack([np.array([rng.integers(-1, i) if i else -1 for i in range(T)]) for _ in range(B)])
    chain = rng.random((B, T)) < 0.4
    return np.where(chain, np.arange(T)[None] - 1, p)


def ancestors(parents):
    """Words by walking up, one draft at a time, as signed 64-bit numbers."""
    out = np.zeros(parents.shape, np.int64)
    for b, row in enumerate(parents):
        for i in range(len(row)):
            w, j = 0, i
            while j >= 0:
                w |= 1 << j
                j = int(row[j])
            out[b, i] = w - 2 ** 64 if w >= 2 ** 63 else w
    return out
