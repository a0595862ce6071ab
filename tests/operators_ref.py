"""Plain float64 (numpy) definitions of the operators around the decode step: rotary positions, causal
attention with its log-sum-exp over packed or paged rows, accumulated attention weights, eviction."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim, base=10000.0, method="none", factor=1.0, original_context=0, slow_turns=1.0, fast_turns=None):
    """Radians per position of each pair, and the factor on cos and sin."""
    out, magnitude = [], 0.1 * math.log(factor) + 1.0 if method == "ramp" else 1.0
    fast = fast_turns if fast_turns is not None else (32.0 if method == "ramp" else 4.0)
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        turns = original_context * f / (2 * math.pi)  # over the original context
        if method == "linear":
            f /= factor
        elif method == "base":
            f = (base * factor ** (rotary_dim / (rotary_dim - 2))) ** (-2.0 * i / rotary_dim)
        elif method == "bands":
            w = min(max((turns - slow_turns) / (fast - slow_turns), 0.0), 1.0)
            f = f * w + f / factor * (1 - w)
        elif method == "ramp":
            index = lambda n: rotary_dim * math.log(original_context / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow_turns)), rotary_dim - 1)
            w = 1 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * w + f / factor * (1 - w)
        out.append(f)
    return np.array(out), magnitude


def rotate(x, positions, freq, magnitude=1.0, interleaved=False):
    """x [T, H, D] float64 -> (rotated, |x_a| + |x_b| of each element's pair, zero where it is copied)."""
    y, size = x.copy(), np.zeros_like(x)
    r = 2 * len(freq)
    a, b = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    angle = positions.astype(np.float64)[:, None] * freq[None]
    c, s = (magnitude * f(angle)[:, None, :] for f in (np.cos, np.sin))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = magnitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def rows_of(cache, table, n):
    """The first n positions of a request: [n, Hkv, D] float64."""
    bs = cache.shape[2]
    out = np.empty((n, cache.shape[1], cache.shape[3]))
    for i in range(0, n, bs):
        m = min(bs, n - i)
        out[i:i + m] = cache[table[i // bs], :, :m].transpose(1, 0, 2)
    return out


def weights(q, k, scale):
    """q [c, Hq, D], the last c of the positions of k [n, Hkv, D]: (p [c, Hq, n], lse [c, Hq]), causal."""
    c, hq, _ = q.shape
    n, hkv, _ = k.shape
    s = np.einsum("chd,nhd->chn", q.astype(np.float64), np.repeat(k, hq // hkv, axis=1)) * scale
    seen = np.arange(n)[None, :] <= (n - c + np.arange(c))[:, None]
    s = np.where(seen[:, None, :], s, -np.inf)
    top = s.max(-1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(-1, keepdims=True)
    return e / total, (top + np.log(total))[..., 0]


def attend(q, k, v, scale):
    """(out [c, Hq, D], lse [c, Hq]); keys a row may not see do not enter it, whatever they hold."""
    p, lse = weights(q, k, scale)
    rep = q.shape[1] // k.shape[1]
    vv = np.repeat(v, rep, axis=1)
    return np.einsum("chn,nhd->chd", p, vv), lse


def evict_positions(scores, n, budget, recent, sinks):
    """The kept positions of one row, ascending."""
    if n <= budget:
        return np.arange(n)
    value = np.where(np.isnan(scores[:n]), -np.inf, scores[:n].astype(np.float64))
    rank = sorted(range(sinks, n - recent), key=lambda t: (np.isnan(scores[t]), -value[t], t))
    keep = list(range(sinks)) + list(range(n - recent, n)) + rank[:budget - recent - sinks]
    return np.array(sorted(keep), dtype=np.int64)


def evict(k_cache, v_cache, scores, tables, new_tables, lens, budget, recent, sinks):
    """(k_cache, v_cache, kept, new_scores, new_lens) after the call."""
    b, hkv, _ = scores.shape
    bs = k_cache.shape[2]
    out = [k_cache.copy(), v_cache.copy()]
    kept = np.full((b, hkv, budget), -1, np.int32)
    new_scores = np.zeros_like(scores)
    for i in range(b):
        for h in range(hkv):
            p = evict_positions(scores[i, h], int(lens[i]), budget, recent, sinks)
            kept[i, h, :len(p)] = p
            new_scores[i, h, :len(p)] = scores[i, h, p]
            for j, t in enumerate(p):
                for old, new in zip((k_cache, v_cache), out):
                    new[new_tables[i, j // bs], h, j % bs] = old[tables[i, t // bs], h, t % bs]
    return out[0], out[1], kept, new_scores, np.minimum(lens, budget).astype(np.int32)
