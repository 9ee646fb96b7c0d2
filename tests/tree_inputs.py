"""Seeded inputs of the drafted-tree tests: random trees, ragged batches over
a scattered pool, and the caches' types."""
import numpy as np
import torch

from oracle.cache_ops import fp8_quantize_rows, int8_quantize_rows
from paged_kv_cache_191_gb300 import workloads as W

KV = {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8}


def parents_of(rng, n, reach=6):
    return np.array([-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, n)], dtype=np.int32)[:n]


def random_mask(rng, n, words):
    """Any visibility, the first row seeing nothing and the last everything."""
    bits = rng.random((n, words * 64)) < 0.4
    if n:
        bits[0] = False
        bits[-1] = True
    return (bits.reshape(n, words, 64).astype(np.uint64) << np.arange(64, dtype=np.uint64)).sum(
        -1, dtype=np.uint64).view(np.int64).reshape(n, words)


def quantised(rng, blocks, Hkv, D, kind):
    """A pool of 1-byte codes with its per-token scales, and nothing else."""
    x = rng.standard_normal((blocks * 16, Hkv, D)).astype(np.float32)
    codes, scale = (int8_quantize_rows if kind == "int8" else fp8_quantize_rows)(x)
    codes = codes.reshape(blocks, 16, Hkv, D).transpose(0, 2, 1, 3)
    return np.ascontiguousarray(codes), np.ascontiguousarray(scale.reshape(blocks, 16))


class TreeBatch:
    """Queries, tables, lengths, masks and a pool of one ragged batch."""

    def __init__(self, seed, Hq, Hkv, D, kind, sizes, lens, q_dtype=None, masks="tree"):
        rng = W.rng_for(seed)
        self.kind, self.D, self.Hq, self.Hkv = kind, D, Hq, Hkv
        self.sizes, self.lens = np.array(sizes, dtype=np.int64), np.array(lens, dtype=np.int32)
        self.q_start = np.concatenate([[0], np.cumsum(self.sizes)]).astype(np.int32)
        T = int(self.q_start[-1])
        nblk = -(-self.lens.astype(np.int64) // 16)
        blocks = int(nblk.sum()) + 3
        order = rng.permutation(blocks).astype(np.int64)
        self.tables = W._tables_from_order(order, self.lens, max(1, int(nblk.max(initial=1))))
        self.words = max(1, -(-int(self.sizes.max(initial=0)) // 64))
        self.parents = [parents_of(rng, int(n)) for n in self.sizes]
        rows = []
        for n, par in zip(self.sizes, self.parents):
            if masks == "tree":
                m = np.zeros((n, self.words), dtype=np.uint64)
                for i in range(n):
                    if par[i] >= 0:
                        m[i] = m[par[i]]
                    m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
                rows.append(m.view(np.int64))
            else:
                rows.append(random_mask(rng, int(n), self.words))
        self.mask = np.concatenate(rows) if rows else np.zeros((0, self.words), np.int64)
        qdt = q_dtype or (KV[kind] if kind in ("f16", "bf16") else torch.float16)
        self.q = W.randn(rng, (T, Hq, D), qdt)
        self.k_scale = self.v_scale = None
        if kind in ("fp8", "int8"):
            (k, ks), (v, vs) = quantised(rng, blocks, Hkv, D, kind), quantised(rng, blocks, Hkv, D, kind)
            self.k, self.v = torch.from_numpy(k), torch.from_numpy(v)
            self.k_scale, self.v_scale = torch.from_numpy(ks), torch.from_numpy(vs)
        else:
            self.k = W.randn(rng, (blocks, Hkv, 16, D), KV[kind])
            self.v = W.randn(rng, (blocks, Hkv, 16, D), KV[kind])
        self.scale = D ** -0.5
