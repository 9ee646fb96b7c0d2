"""Cases of decoding over a block-scaled cache, and of sampled verification.

  append   this step's K and V rows into a cache of E4M3 codes that has one
           power-of-two scale for every (block, kv head)
  attend   attention over that cache: single tokens, drafted chains, prompt
           chunks (causal among a sequence's new tokens)
  verify   drafted tokens against the target's probabilities, from given random
           numbers: the accepted path and the token drawn behind it

``listed`` and ``draw`` give the cases, ``prepare`` a case's inputs, ``run``
one pass through its operator: in plain torch, or through the package where
``own`` is true.  A sequence's new tokens are the last n_b of its context.
"""
import math

import numpy as np
import torch

own = False

BLOCK, DIM, MOST = 16, 128, 448.0  # tokens of a block, head_dim, the largest E4M3 value
KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one user's next token enters the cache: latency
        dict(name="append_token", op="append", B=1, Hq=32, Hkv=8, dtype="f16", n_lo=1, n_hi=1, len_lo=600, len_hi=600),
        # the decode step of the grouped-query batch of 64
        dict(name="append_step", op="append", B=64, Hq=64, Hkv=8, dtype="bf16", n_lo=1, n_hi=1, len_lo=16, len_hi=4096),
        # prompts of odd lengths beside drafted chains, multi-head shape
        dict(name="append_prompts", op="append", B=9, Hq=32, Hkv=32, dtype="f16", n_lo=3, n_hi=2043, len_lo=2043,
             len_hi=2100),
        # one user's next token over a short context: latency
        dict(name="attend_token", op="attend", B=1, Hq=32, Hkv=8, dtype="f16", n_lo=1, n_hi=1, len_lo=600, len_hi=600),
        # the multi-head batch of 32, ragged contexts up to 2048
        dict(name="attend_mha_step", op="attend", B=32, Hq=32, Hkv=32, dtype="f16", n_lo=1, n_hi=1, len_lo=1,
             len_hi=2048),
        # the grouped-query batch of 64
        dict(name="attend_gqa_step", op="attend", B=64, Hq=64, Hkv=8, dtype="bf16", n_lo=1, n_hi=1, len_lo=16,
             len_hi=4096),
        # long contexts
        dict(name="attend_long_step", op="attend", B=8, Hq=32, Hkv=8, dtype="f16", n_lo=1, n_hi=1, len_lo=16384,
             len_hi=32768),
        # drafted chains of up to 5 tokens are checked in the grouped-query batch
        dict(name="attend_chains", op="attend", B=64, Hq=64, Hkv=8, dtype="bf16", n_lo=2, n_hi=5, len_lo=16,
             len_hi=4096),
        # prompt chunks behind their contexts: the most arithmetic
        dict(name="attend_prompts", op="attend", B=4, Hq=32, Hkv=8, dtype="f16", n_lo=300, n_hi=1024, len_lo=1024,
             len_hi=4096),
        # one user's chain of 4 drafted tokens: latency
        dict(name="verify_chain", op="verify", B=1, n_lo=5, n_hi=5, V=32000, drafts="sampled"),
        # a full batch's chains over a large vocabulary
        dict(name="verify_batch", op="verify", B=256, n_lo=3, n_hi=9, V=128000, drafts="sampled"),
        # trees whose nodes are picked without a draft distribution, a vocabulary of odd size
        dict(name="verify_trees", op="verify", B=48, n_lo=9, n_hi=26, V=65521, drafts="tree"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "verify"])
    most = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        if op == "verify":
            drafts = rng.choice(["sampled", "picked", "tree"])
            n_hi = _log(rng, 1, 32 if drafts == "tree" else 12)
            c = dict(op=op, B=_log(rng, 1, 256), n_lo=rng.randint(1, n_hi), n_hi=n_hi, V=_log(rng, 200, 131072),
                     drafts=drafts)
            if c["B"] * (c["n_lo"] + n_hi) // 2 * c["V"] > 200e6:
                continue
        else:
            Hkv = rng.choice([1, 2, 4, 8, 16, 32])
            Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 6, 8) if g * Hkv <= 64])
            n_hi = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)])
            len_hi = max(n_hi, _log(rng, 1, 32768))
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv,
                     dtype=rng.choice(["f16", "bf16", "f32"] if op == "append" else ["f16", "bf16"]),
                     n_lo=rng.randint(max(1, n_hi // 3), n_hi), n_hi=n_hi, len_lo=rng.randint(n_hi, len_hi), len_hi=len_hi)
            pool = c["B"] * len_hi * Hkv * DIM * 4
            scores = c["B"] * Hq * n_hi * len_hi * 4 if op == "attend" else 0
            if pool > 2 << 30 or scores > 3 << 30:
                continue
        w = work(c)
        if all(w[k] <= most[k] for k in most):
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread: every seed has the same ones, in another order."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def work(case):
    c = case
    n = _spread(c["n_lo"], c["n_hi"], c["B"])
    T, B = int(n.sum()), c["B"]
    if c["op"] == "verify":
        rows = 2 if c["drafts"] == "sampled" else 1  # the row drawn from, and its draft's
        return {"bytes": B * c["V"] * 4 * rows + T * 24 + B * (4 * c["n_hi"] + 16), "flops": B * c["V"] * 3}
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": T * c["Hkv"] * 2 * DIM * (size + 1) + (T // BLOCK + 1) * c["Hkv"] * 8,
                "flops": T * c["Hkv"] * 2 * DIM * 3}
    L = _spread(c["len_lo"], c["len_hi"], B)
    kv = int(L.sum()) * c["Hkv"] * 2 * DIM + int((-(-L // BLOCK)).sum()) * (c["Hkv"] * 8 + 4)
    return {"bytes": kv + T * c["Hq"] * DIM * 4,
            "flops": 4 * DIM * c["Hq"] * int((n * (L - n) + n * (n + 1) // 2).sum())}


# ---- inputs ----------------------------------------------------------------
def prepare(case, seed):
    c = case
    rng = np.random.Generator(np.random.PCG64(seed))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    B = c["B"]
    n = rng.permutation(_spread(c["n_lo"], c["n_hi"], B))
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(q_start[-1])
    s = {"case": c, "q_start": dev(q_start), "max_n": int(n.max())}
    if c["op"] == "verify":
        V = c["V"]
        logits = randn(T, V).mul_(3.0)
        s["target"] = torch.softmax(logits, -1)
        if c["drafts"] == "sampled":
            draft = torch.softmax(logits.add_(randn(T, V)), -1)
        del logits
        # a node's parent: the node before it, or any of the six before it
        parents = np.concatenate([np.arange(k) - 1 for k in n])
        if c["drafts"] == "tree":
            parents = np.concatenate([[-1, *(int(rng.integers(max(0, i - 6), i)) for i in range(1, k))] for k in n])
        at = dev(np.maximum(np.repeat(q_start[:-1], n) + parents, 0))
        noise = torch.rand((T, V), generator=gen, device="cuda").log_().neg_()  # exponential: argmax p / e draws from p
        s["tokens"] = noise.reciprocal_().mul_((draft if c["drafts"] == "sampled" else s["target"])[at]).argmax(-1)
        s["draft"] = draft if c["drafts"] == "sampled" else None
        s["parents"] = dev(parents.astype(np.int32)) if c["drafts"] == "tree" else None
        s["uniform"] = torch.rand((T,), generator=gen, device="cuda")
        return s
    L = rng.permutation(_spread(c["len_lo"], c["len_hi"], B))
    nblk = -(-L // BLOCK)
    blocks = int(nblk.sum()) + 3
    order = rng.permutation(blocks)
    tables = np.full((B, int(nblk.max())), -1, dtype=np.int32)
    tables[np.arange(tables.shape[1])[None] < nblk[:, None]] = order[:int(nblk.sum())]
    code = lambda: (randn(blocks, c["Hkv"], BLOCK, DIM, dtype=torch.float16) * 90).clamp_(-MOST, MOST).to(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: 2.0 ** -torch.randint(6, 9, (blocks, c["Hkv"]), generator=gen, device="cuda").float()  # noqa: E731
    s |= {"tables": dev(tables), "lens": dev(L.astype(np.int32)), "max_len": int(L.max()), "k_cache": code(),
          "v_cache": code(), "k_scale": scale(), "v_scale": scale()}
    # the projections' output, queries, keys and values of a token side by side
    qkv = randn(T, (c["Hq"] + 2 * c["Hkv"]) * DIM, dtype=KINDS[c["dtype"]]).unflatten(1, (-1, DIM))
    s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
    return s


# ---- one pass --------------------------------------------------------------
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_191_gb300 import ops
        if op == "append":
            ops.block_scaled_append(s["k"], s["v"], s["q_start"], s["tables"], s["lens"], s["k_cache"], s["v_cache"],
                                    s["k_scale"], s["v_scale"])
            return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}
        if op == "attend":
            return ops.block_scaled_attention(s["q"], s["q_start"], s["k_cache"], s["v_cache"], s["k_scale"],
                                              s["v_scale"], s["tables"], s["lens"], s["max_len"], s["max_n"],
                                              DIM ** -0.5)
        path, count, token = ops.draft_verify(s["tokens"], s["target"], s["uniform"], s["q_start"], s["max_n"],
                                              draft_probs=s["draft"], parents=s["parents"])
        return {"path": path, "path_len": count, "next_token": token}
    return {"append": _append, "attend": _attend, "verify": _verify}[op](s)


def _append(s):
    start, L = s["q_start"].long(), s["lens"].long()
    count = start.diff()
    first = L - count  # position of a sequence's first new token
    # the blocks that get rows, as many for every sequence (its last one again where it has fewer)
    j = torch.arange((s["max_n"] + 2 * BLOCK - 2) // BLOCK, device=L.device)
    j = torch.minimum((first // BLOCK)[:, None] + j, ((L - 1) // BLOCK)[:, None])
    block = torch.gather(s["tables"].long(), 1, j)
    pos = j[..., None] * BLOCK + torch.arange(BLOCK, device=L.device)  # [B, J, 16]
    new = (pos >= first[:, None, None]) & (pos < L[:, None, None])
    kept = pos < first[:, None, None]
    at = (start[:-1, None, None] + pos - first[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[at].float().transpose(2, 3)  # [B, J, Hkv, 16, D]
        size = x.abs()
        size = torch.where((size < math.inf) & new[:, :, None, :, None], size, 0.0).amax((3, 4))
        # the smallest power of two that brings the largest value to at most 448 = 0.875 x 2^9
        mant, exp = torch.frexp(size)
        want = torch.ldexp(torch.ones_like(size), (exp - 9 + (mant > 0.875)).clamp(min=-126))
        old = torch.where(kept.any(2)[..., None], scale[block], 0.0)
        top = torch.maximum(torch.where(size > 0, want, 0.0), old)
        top = torch.where(top > 0, top, 1.0)
        code = cache[block].float()
        less = torch.where(kept[:, :, None, :, None], (old / top)[..., None, None], 1.0)  # rows that stay, under a larger scale
        code = torch.where(new[:, :, None, :, None], (x / top[..., None, None]).clamp(-MOST, MOST), code * less)
        cache[block] = code.to(torch.float8_e4m3fn)
        scale[block] = top
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _attend(s):
    c = s["case"]
    T, Hq, _ = s["q"].shape
    N, G = s["max_n"], Hq // c["Hkv"]
    start, count, L = s["q_start"][:-1].long(), s["q_start"].diff().long(), s["lens"].long()
    node = torch.arange(N, device=L.device)
    live = node[None] < count[:, None]
    at = (start[:, None] + node[None]).clamp(max=T - 1)
    blocks = s["tables"].clamp(min=0).long()
    K, V = ((s[x][blocks].float() * s[y][blocks][..., None, None]).transpose(1, 2).flatten(2, 3)
            for x, y in (("k_cache", "k_scale"), ("v_cache", "v_scale")))  # [B, Hkv, tokens, D]
    t = torch.arange(K.shape[2], device=L.device)
    sees = live[..., None] & (t <= (L - count)[:, None, None] + node[None, :, None])
    q = s["q"][at].float().unflatten(2, (c["Hkv"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, N G, D]
    x = (q @ K.transpose(2, 3)).unflatten(2, (N, G)) * DIM ** -0.5
    x = x.masked_fill(~sees[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    V = V.masked_fill((t[None] >= L[:, None])[:, None, :, None], 0.0)
    out = (p.flatten(2, 3) @ V).unflatten(2, (N, G)) / total.clamp(min=1e-30)
    return out.permute(0, 2, 1, 3, 4).flatten(2, 3)[live].to(s["q"].dtype)


def _verify(s):
    N, T = s["max_n"], s["tokens"].numel()
    start, count = s["q_start"][:-1].long(), s["q_start"].diff().long()
    node = torch.arange(N, device=start.device)
    live = node[None] < count[:, None]
    at = (start[:, None] + node[None]).clamp(max=T - 1)
    parent = node[None] - 1 if s["parents"] is None else s["parents"][at].long()
    parent = torch.where(live, parent, -1)
    token, u = s["tokens"][at], s["uniform"][at].double()
    row = (start[:, None] + parent.clamp(min=0)).clamp(max=T - 1)
    p = s["target"][row, token].double()
    child = live & (parent >= 0)
    # siblings before a node: their tokens were refused, and their share is gone
    older = (parent[:, :, None] == parent[:, None]) & child[:, None] & (node[None, :] < node[:, None])
    same = older & (token[:, :, None] == token[:, None])
    fresh = child & ~same.any(-1)  # (a token refused once has nothing left)
    rest = 1.0 - (older & fresh[:, None]).double().mul(p[:, None]).sum(-1)
    q = rest if s["draft"] is None else s["draft"][row, token].double()
    hit = fresh & (u * q < p)
    hit = hit & ~(older & hit[:, None]).any(-1)
    # a node's ancestors by powers of "is the parent of": all of them have to be hit
    up = (parent[:, :, None] == node).float() + torch.eye(N, device=start.device)
    reach = torch.linalg.matrix_power(up, N) > 0
    taken = live & ((~reach) | (hit | (node == 0))[:, None]).all(-1)
    path_len = taken.sum(1)
    path = torch.full((len(start), N + 1), -1, dtype=torch.int64, device=start.device)
    path.scatter_(1, torch.where(taken, taken.cumsum(1) - 1, N), node.expand(len(start), -1))
    path[:, N] = -1
    last = torch.gather(path, 1, (path_len - 1).clamp(min=0)[:, None])
    whole = s["target"][(start + last[:, 0].clamp(min=0)).clamp(max=T - 1)].double()  # the row drawn from
    left = whole.clone()
    refused = child & (parent == last)
    if s["draft"] is None:
        # (tokens of other nodes keep what they have)
        left.scatter_reduce_(1, token, torch.where(refused, 0.0, 2.0).double(), "amin")
    else:
        left -= s["draft"][(start + last[:, 0].clamp(min=0)).clamp(max=T - 1)].double() * refused.any(1)[:, None]
    sums = left.clamp_(min=0).cumsum(1)
    # (a draft that leaves nothing: the target's row as it is)
    sums = torch.where(sums[:, -1:] > 0, sums, whole.cumsum(1))
    drawn = torch.searchsorted(sums, u[:, :1] * sums[:, -1:], right=True)[:, 0].clamp(max=sums.shape[1] - 1)
    return {"path": path[:, :N].int().contiguous(), "path_len": path_len.int(),
            "next_token": torch.where(path_len > 0, drawn, -1)}


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    """Codes and scales one block at a time, attention one sequence at a time.  Paths and tokens are not computed
    numbers."""
    s = prepare(case, seed)
    c = case
    starts, lens = s["q_start"].tolist(), (s["lens"].tolist() if "lens" in s else [])
    if c["op"] == "verify":
        return None
    if c["op"] == "append":
        if c["B"] * c["n_hi"] > 40000:  # (a loop over blocks)
            return None
        return _exact_append(s, starts, lens)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b, L in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        at = s["tables"][b, :-(-L // BLOCK)].long()
        reach = torch.arange(L - (hi - lo), L, device="cuda")  # the last key that each token sees
        hidden = torch.arange(L, device="cuda")[None] > reach[:, None]
        for g in range(c["Hkv"]):
            K, V = ((s[x][at, g].double() * s[y][at, g].double()[:, None, None]).flatten(0, 1)[:L]
                    for x, y in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
            x = torch.einsum("nhd,ld->hnl", s["q"][lo:hi, g * G:(g + 1) * G].double(), K) / math.sqrt(DIM)
            w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[lo:hi, g * G:(g + 1) * G] = torch.einsum("hnl,ld->nhd", w, V)
    return out


def _round_e4m3(x):
    """x to the nearest E4M3 value, ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-MOST, MOST)


def _exact_append(s, starts, lens):
    out = {x: s[x].double() for x in ("k_cache", "v_cache", "k_scale", "v_scale")}
    tables = s["tables"].tolist()
    for b, L in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        p0 = L - (hi - lo)
        for j in range(p0 // BLOCK, -(-L // BLOCK)):
            blk, a, e = tables[b][j], max(p0, j * BLOCK), min(L, (j + 1) * BLOCK)
            r0 = a - j * BLOCK
            for x, cache, scale in ((s["k"], "k_cache", "k_scale"), (s["v"], "v_cache", "v_scale")):
                rows = x[lo + a - p0:lo + e - p0].double().transpose(0, 1)  # [Hkv, new, D]
                need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / MOST)))
                new = torch.maximum(need, out[scale][blk]) if r0 else need
                code = out[cache][blk]
                if r0:
                    code[:, :r0] = _round_e4m3(code[:, :r0] * (out[scale][blk] / new)[:, None, None])
                code[:, r0:r0 + e - a] = _round_e4m3(rows / new[:, None, None])
                out[scale][blk] = new
    return out
