"""The drafted-tree step by its definition (test infrastructure only).

[LLM-INF] section 6.1 has the target model check the draft's tokens in one
pass.  Here the draft is a tree: the last n_b tokens of sequence b's context
are its nodes, node 0 the current token, every other node below an earlier one.
Readings where the pages are silent:

* rotary positions: pair i of a head's first rot dims turns by position *
  inv_freq[i], cosine and sine times one factor; pairs are dims (i, i + rot/2),
  or (2 i, 2 i + 1) when interleaved;
* node i sees every key of the context before the tree and the nodes whose
  bits its mask row sets; a row that sees no key is zero;
* acceptance is token matching: after an accepted node comes its lowest child
  whose drafted token is the one the model picked after the node;
* the accepted nodes' rows are moved to the front of the tree's positions.
"""
import numpy as np

from .attention import BLOCK_SIZE, gather_kv


def rotate(x, positions, inv_freq, factor=1.0, interleaved=False):
    """x [T, H, D] rotated, float64, and per value the sum of the two products'
    magnitudes (what a rounding error of the rotation is relative to)."""
    x = np.asarray(x).astype(np.float64)
    rot = 2 * len(inv_freq)
    # the angle modulo one turn, in extended precision: far positions turn many times
    turns = np.asarray(positions, dtype=np.longdouble)[:, None] * (
        np.asarray(inv_freq, dtype=np.longdouble) / (2 * np.arctan2(np.longdouble(0), np.longdouble(-1))))
    a = ((turns - np.floor(turns)) * 2).astype(np.float64) * np.pi
    c, s = (factor * f(a)[:, None, :] for f in (np.cos, np.sin))
    out, mag = x.copy(), np.abs(x)
    i1 = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    i2 = i1 + 1 if interleaved else i1 + rot // 2
    x1, x2 = x[..., i1], x[..., i2]
    out[..., i1], out[..., i2] = x1 * c - x2 * s, x1 * s + x2 * c
    mag[..., i1] = mag[..., i2] = (np.abs(x1) + np.abs(x2)) * abs(factor)
    return out, mag


def visible(mask_row, n):
    """Bits 0 .. n - 1 of a row of int64 words."""
    words = np.asarray(mask_row).view(np.uint64)
    j = np.arange(n)
    return ((words[j // 64] >> (j % 64).astype(np.uint64)) & np.uint64(1)).astype(bool)


def tree_attention(q, q_start, mask, k_cache, v_cache, tables, lens, scale, k_scale=None, v_scale=None):
    """(out, spread, score) float64: out [T, Hq, D]; spread [T, Hq, D] =
    sum_t w_t |V_t| and score [T, Hq] = max_t sum_d |scale q_d K_td| over the
    keys seen, the magnitudes that rounding errors are relative to."""
    q = np.asarray(q).astype(np.float64)
    T, Hq, D = q.shape
    G = Hq // k_cache.shape[1]
    out, spread, score = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b, L in enumerate(int(x) for x in lens):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        n = hi - lo
        for g in range(Hq // G):
            K = gather_kv(k_cache, tables[b], L, g, k_scale)
            V = gather_kv(v_cache, tables[b], L, g, v_scale)
            for i in range(n):
                sees = np.ones(L, dtype=bool)
                t = np.arange(max(0, L - n), L)  # the nodes that are cached
                sees[t] = visible(mask[lo + i], n)[t - (L - n)]
                if not sees.any():
                    continue
                Ks, Vs = K[sees], V[sees]
                for h in range(g * G, (g + 1) * G):
                    s = scale * (Ks @ q[lo + i, h])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[lo + i, h] = w @ Vs
                    spread[lo + i, h] = w @ np.abs(Vs)
                    score[lo + i, h] = abs(scale) * (np.abs(Ks) @ np.abs(q[lo + i, h])).max()
    return out, spread, score


def tree_largest(q, q_start, mask, k_cache, tables, lens, scale, k_scale=None, v_scale=None):
    """float64 [T, Hq]: the largest softmax weight of a row, times its key's V scale."""
    q = np.asarray(q).astype(np.float64)
    T, Hq, _ = q.shape
    G = Hq // k_cache.shape[1]
    most = np.zeros((T, Hq))
    for b, L in enumerate(int(x) for x in lens):
        lo, n = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b])
        t = np.arange(L)
        vs = np.ones(L) if v_scale is None else np.abs(v_scale[tables[b][t // BLOCK_SIZE], t % BLOCK_SIZE]).astype(np.float64)
        for g in range(Hq // G):
            K = gather_kv(k_cache, tables[b], L, g, k_scale)
            for i in range(n):
                sees = np.ones(L, dtype=bool)
                nodes = np.arange(max(0, L - n), L)
                sees[nodes] = visible(mask[lo + i], n)[nodes - (L - n)]
                for h in range(g * G, (g + 1) * G):
                    s = scale * (K[sees] @ q[lo + i, h])
                    w = np.exp(s - s.max(initial=-np.inf))
                    most[lo + i, h] = (w * vs[sees]).max(initial=0.0) / max(w.sum(), 1e-300)
    return most


def tree_accept(draft, target, parents, q_start, max_path):
    """(paths, next tokens): lists per sequence."""
    paths, tokens = [], []
    for lo, hi in zip(q_start[:-1], q_start[1:]):
        path = [0] if hi > lo else []
        while path and len(path) < max_path:
            cur = path[-1]
            kids = [i for i in range(cur + 1, hi - lo)
                    if parents[lo + i] == cur and draft[lo + i] == target[lo + cur]]
            if not kids:
                break
            path.append(kids[0])
        paths.append(path)
        tokens.append(int(target[lo + path[-1]]) if path else -1)
    return paths, tokens


def tree_commit(caches, tables, lens, q_start, paths):
    """(new caches, new lengths): every array of `caches` ([blocks, Hkv, 16, D]
    rows or [blocks, 16] scales) with the paths' rows moved."""
    new = [np.array(c, copy=True) for c in caches]
    out = []
    for b, path in enumerate(paths):
        first = int(lens[b]) - int(q_start[b + 1] - q_start[b])
        for i, p in enumerate(path):
            src, dst = first + p, first + i
            s, d = (int(tables[b][src // BLOCK_SIZE]), src % BLOCK_SIZE), (int(tables[b][dst // BLOCK_SIZE]), dst % BLOCK_SIZE)
            for old, c in zip(caches, new):
                if old.ndim == 4:
                    c[d[0], :, d[1]] = old[s[0], :, s[1]]
                else:
                    c[d] = old[s]
        out.append(first + len(path))
    return new, out
