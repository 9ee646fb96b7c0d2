"""Block-scaled caches and sampled verification by their definitions (test
infrastructure only).

[LLM-INF] section 5.3 names FP8 caches with per-token or per-channel scales;
here a scale belongs to a (block, kv head) tile of 16 tokens.  Section 6.1
verifies drafted tokens in one pass.  Readings where the pages are silent:

* a scale is the smallest power of two (not below 2^-126) that brings the new
  finite values to at most 448; rows that stay in the block keep it from
  shrinking, and are rounded to it when it grows; a block whose first row is
  new starts afresh, with scale 1 if it has no value above 0;
* a token at position t sees the keys 0 .. t;
* refused siblings' tokens have nothing left; weights are whole multiples of
  2^-44, to nearest even.
"""
import math
from fractions import Fraction

import numpy as np

from .fp8_e4m3 import e4m3_decode, e4m3_encode

BLOCK, D = 16, 128


def power_scale(x):
    """Smallest power of two s >= 2^-126 with |x| <= 448 s, 0 for none."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    top = float(a[np.isfinite(a)].max(initial=0.0))
    if top == 0.0:
        return 0.0
    e = -126
    while math.ldexp(448.0, e) < top:
        e += 1
    return math.ldexp(1.0, e)


def append(k_cache, v_cache, k_scale, v_scale, k, v, q_start, tables, lens):
    """New (k_cache, v_cache, k_scale, v_scale); codes uint8 [nb, Hkv, 16, D]."""
    out = [np.array(x, copy=True) for x in (k_cache, v_cache, k_scale, v_scale)]
    for b, L in enumerate(int(x) for x in lens):
        lo, n = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b])
        first = L - n
        for j in range(first // BLOCK, -(-L // BLOCK) if n else 0):
            blk, r0, r1 = int(tables[b][j]), max(0, first - j * BLOCK), min(BLOCK, L - j * BLOCK)
            at = lo + j * BLOCK + r0 - first
            for cache, scale, x in ((out[0], out[2], k), (out[1], out[3], v)):
                for g in range(cache.shape[1]):
                    new = np.asarray(x[at:at + r1 - r0, g], dtype=np.float64)
                    old = float(scale[blk, g]) if r0 else 0.0
                    s = max(power_scale(new), old) or 1.0
                    if r0 and s > old:
                        cache[blk, g, :r0] = e4m3_encode(e4m3_decode(cache[blk, g, :r0]) * (old / s))
                    cache[blk, g, r0:r1] = e4m3_encode(new / s)
                    scale[blk, g] = s
    return out


def gather(cache, scale, table, L, g):
    """The first L rows of one kv head, float64 [L, D]."""
    nb = -(-L // BLOCK)
    ids = np.asarray(table[:nb], dtype=np.int64)
    x = e4m3_decode(cache[ids, g]) * np.asarray(scale, dtype=np.float64)[ids, g][:, None, None]
    return x.reshape(nb * BLOCK, cache.shape[-1])[:L]


def attention(q, q_start, k_cache, v_cache, k_scale, v_scale, tables, lens, scale):
    """(out, spread, score, wide) float64: out [T, Hq, D]; spread = sum_t w_t
    |V_t|; score [T, Hq] = max_t sum_d |scale q_d K_td| and wide = max_t |scale|
    max |q| sum_d |K_td|: the magnitudes that errors are relative to."""
    q = np.asarray(q).astype(np.float64)
    T, Hq, _ = q.shape
    G = Hq // k_cache.shape[1]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    score, wide = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b, L in enumerate(int(x) for x in lens):
        lo, n = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b])
        for g in range(Hq // G):
            K, V = gather(k_cache, k_scale, tables[b], L, g), gather(v_cache, v_scale, tables[b], L, g)
            for i in range(n):
                m = L - n + i + 1
                if m <= 0:
                    continue
                x = q[lo + i, g * G:(g + 1) * G]
                s = scale * (x @ K[:m].T)
                w = np.exp(s - s.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                h = slice(g * G, (g + 1) * G)
                out[lo + i, h] = w @ V[:m]
                spread[lo + i, h] = w @ np.abs(V[:m])
                score[lo + i, h] = (np.abs(scale * x) @ np.abs(K[:m]).T).max(axis=1)
                wide[lo + i, h] = abs(scale) * np.abs(x).max(axis=1) * np.abs(K[:m]).sum(axis=1).max()
    return out, spread, score, wide


def fixed(p):
    """Probabilities as whole multiples of 2^-44, to nearest even."""
    p = np.asarray(p, dtype=np.float64)
    return np.rint(np.clip(np.where(np.isnan(p), 0.0, p), 0.0, 1.0) * 2.0 ** 44).astype(np.int64).astype(object)


def verify(tokens, target, uniform, q_start, max_path, draft=None, parents=None):
    """(paths, next tokens): lists, one entry per sequence."""
    clip = lambda x: float(np.clip(np.nan_to_num(np.float64(x), nan=0.0), 0.0, 1.0))  # noqa: E731
    V = np.asarray(target).shape[1]
    paths, nexts = [], []
    for b in range(len(q_start) - 1):
        lo, n = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b])
        if n == 0:
            paths.append([])
            nexts.append(-1)
            continue
        par = [-1] + list(range(n - 1)) if parents is None else [int(x) for x in parents[lo:lo + n]]
        tok = [int(x) for x in tokens[lo:lo + n]]
        path, refused = [0], []
        while len(path) < max_path:
            cur, rest, refused, hit = path[-1], 1.0, [], None
            for c in range(cur + 1, n):
                if par[c] != cur:
                    continue
                x = tok[c]
                if 0 <= x < V and x not in refused:
                    p = clip(target[lo + cur, x])
                    q = rest if draft is None else clip(draft[lo + cur, x])
                    if float(uniform[lo + c]) * q < p:
                        hit = c
                        break
                    rest -= p
                refused.append(x)
            if hit is None:
                break
            refused = []
            path.append(hit)
        whole = fixed(target[lo + path[-1]])
        w = whole.copy()
        if refused and draft is not None:
            w = np.maximum(w - fixed(draft[lo + path[-1]]), 0)
        elif refused:
            w[[x for x in refused if 0 <= x < V]] = 0
        if sum(w) == 0:
            w = whole
        total = int(sum(w))
        paths.append(path)
        if total == 0:
            nexts.append(-1)
            continue
        u = float(uniform[lo])
        t = min(math.floor(Fraction(min(u, 1.0)) * total) if u > 0 else 0, total - 1)
        nexts.append(int(np.argmax(np.cumsum(w) > t)))
    return paths, nexts
