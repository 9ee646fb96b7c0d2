"""Seeded inputs of the block-scaled cache's and the verification's tests."""
import numpy as np
import torch

from oracle.scaled import BLOCK, D
from paged_kv_cache_191_gb300 import workloads as W


class ScaledBatch:
    """A ragged batch over a scattered block-scaled pool, new rows and queries."""

    def __init__(self, seed, Hq, Hkv, sizes, lens, dtype=torch.float16, spare=3):
        rng = W.rng_for(seed)
        self.Hq, self.Hkv = Hq, Hkv
        self.sizes, self.lens = np.array(sizes, dtype=np.int64), np.array(lens, dtype=np.int32)
        self.q_start = np.concatenate([[0], np.cumsum(self.sizes)]).astype(np.int32)
        T = int(self.q_start[-1])
        nblk = -(-self.lens.astype(np.int64) // BLOCK)
        blocks = int(nblk.sum()) + spare
        order = rng.permutation(blocks).astype(np.int64)
        self.tables = W._tables_from_order(order, self.lens, max(1, int(nblk.max(initial=1))))
        shape = (blocks, Hkv, BLOCK, D)
        finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
        # (codes near 2^5, as values of a normal distribution under their block's scale are)
        common = np.array([c for c in finite if 0x40 <= (c & 0x7F) <= 0x6F], dtype=np.uint8)
        self.k, self.v = (np.where(rng.random(shape) < 0.05, rng.choice(finite, shape), rng.choice(common, shape))
                          for _ in range(2))
        self.k_scale, self.v_scale = ((2.0 ** -rng.integers(5, 9, (blocks, Hkv))).astype(np.float32) for _ in range(2))
        self.dtype = dtype
        self.new_k, self.new_v = (W.randn(rng, (T, Hkv, D), dtype) for _ in range(2))
        self.q = W.randn(rng, (T, Hq, D), dtype if dtype != torch.float32 else torch.float16)
        self.scale = D ** -0.5


class Drafts:
    """Chains or trees with probabilities of a small or large vocabulary."""

    def __init__(self, seed, sizes, V, kind, sharp=2.0):
        rng = W.rng_for(seed)
        self.q_start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        T = int(self.q_start[-1])
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        logits = sharp * rng.standard_normal((T, V))
        self.target = soft(logits)
        self.draft = soft(logits + rng.standard_normal((T, V))) if kind == "sampled" else None
        self.parents = None
        if kind == "tree":
            self.parents = np.concatenate(
                [np.array([-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)], dtype=np.int32)[:n]
                 for n in sizes] + [np.zeros(0, np.int32)])
        self.tokens = rng.integers(0, V, T)
        for b, n in enumerate(sizes):
            for i in range(1, n):
                at = self.q_start[b] + (i - 1 if self.parents is None else self.parents[self.q_start[b] + i])
                p = (self.draft if self.draft is not None else self.target)[at].astype(np.float64)
                self.tokens[self.q_start[b] + i] = rng.choice(V, p=p / p.sum())
        self.uniform = rng.random(T, dtype=np.float32)
