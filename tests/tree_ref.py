"""Plain float64 (numpy) definitions of the operators around a drafted tree and the fp8 cache's fused append: norms with
the rotation by positions of several axes, trees' masks, attention under a mask, accepted paths."""
from __future__ import annotations

import numpy as np

SCALE = 128 ** -0.5


def norm_rotate(x, weight, eps, positions, axes, freq, magnitude=1.0, interleaved=False):
    """x [T, H, D] float64 -> (normalised and rotated, the size its float32 error goes by).  positions [T, A], axes one
    entry per pair; weight None: no norm."""
    y = x if weight is None else x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
    out, size = y.copy(), np.abs(y)
    r = 2 * len(freq)
    a, b = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    angle = positions.astype(np.float64)[:, axes] * freq[None]
    c, s = (magnitude * f(angle)[:, None, :] for f in (np.cos, np.sin))
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = size[..., b] = magnitude * (np.abs(y[..., a]) + np.abs(y[..., b]))
    return out, size


def ancestors(parents):
    """[n, n] bool: whether node j is node i or above it."""
    n = len(parents)
    seen = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = parents[j]
    return seen


def pack_masks(seen, words):
    """[n, n] bool -> int32 [n, words], bit j % 32 of word j / 32."""
    n = seen.shape[0]
    bits = np.zeros((n, words * 32), np.uint64)
    bits[:, :n] = seen
    packed = (bits.reshape(n, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return packed.astype(np.uint32).view(np.int32)


def rows_of(cache, table, n):
    """The first n positions of a request: [n, Hkv, D]."""
    bs = cache.shape[2]
    p = np.arange(n)
    return cache[table[p // bs], :, p % bs]


def attend(q, k, v, seen, scale=SCALE):
    """q [c, Hq, D], the last c of the positions of k, v [n, Hkv, D]; seen [c, c]: (out, lse, weights [c, Hq, n]).  What a
    row does not see does not enter it, whatever it holds; a row that sees nothing is zero."""
    c, hq, d = q.shape
    n, hkv, _ = k.shape
    whole = np.concatenate([np.ones((c, n - c), bool), seen], 1)
    out, lse, p = np.zeros((c, hq, d)), np.full((c, hq), -np.inf), np.zeros((c, hq, n))
    for i in range(c):
        at = np.nonzero(whole[i])[0]
        if len(at) == 0:
            continue
        for h in range(hq):
            g = h * hkv // hq
            s = k[at, g] @ q[i, h] * scale
            e = np.exp(s - s.max())
            p[i, h, at] = e / e.sum()
            lse[i, h] = s.max() + np.log(e.sum())
            out[i, h] = p[i, h, at] @ v[at, g]
    return out, lse, p
