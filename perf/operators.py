"""Cases of the drafted-tree step over a paged cache: what one speculative
verification step runs between the model's projections and its next step.

  rope    rotary positions of this step's queries and keys, and the store of
          the rotated keys and the values in their cache slots
  tree    attention of every drafted node over its sequence's cached context
          and its own ancestors (the tree mask)
  accept  the accepted path of every sequence's tree, from the tokens the
          model picked after each node
  commit  the accepted nodes' cache rows moved together, behind the context

``listed`` and ``draw`` give the cases, ``prepare`` a case's inputs, ``run``
one pass through its operator: in plain torch, or through the package where
``own`` is true.  A sequence's nodes are the last n_b tokens of its context;
node 0 is its current token, the others hang below an earlier node.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one sequence's tree of 8 nodes enters the cache: latency
        dict(name="rope_small", op="rope", T=8, Hq=32, Hkv=8, D=128, rot=128, dtype="f16", interleaved=False,
             scaling="none", far=4096),
        # a long prompt's tokens, multi-head shape of the batch decode
        dict(name="rope_prompt", op="rope", T=8192, Hq=32, Hkv=32, D=128, rot=128, dtype="f16", interleaved=False,
             scaling="none", far=8192),
        # half of each head rotated in pairs, positions of a long context, an odd number of tokens
        dict(name="rope_far_partial", op="rope", T=1531, Hq=64, Hkv=8, D=128, rot=64, dtype="bf16", interleaved=True,
             scaling="yarn", far=1 << 20),
        # one user's tree over a short context: latency
        dict(name="tree_small", op="tree", B=1, Hq=32, Hkv=8, D=128, dtype="f16", n_lo=8, n_hi=8, len_lo=600,
             len_hi=600),
        # the multi-head batch of 32, ragged contexts up to 2048, small trees of ragged size
        dict(name="tree_mha_batch", op="tree", B=32, Hq=32, Hkv=32, D=128, dtype="f16", n_lo=9, n_hi=26, len_lo=40,
             len_hi=2048),
        # the grouped-query batch of 64 with 16-node trees
        dict(name="tree_gqa_batch", op="tree", B=64, Hq=64, Hkv=8, D=128, dtype="bf16", n_lo=16, n_hi=16, len_lo=32,
             len_hi=4096),
        # long contexts in 1-byte codes
        dict(name="tree_long_fp8", op="tree", B=8, Hq=32, Hkv=8, D=128, dtype="fp8", n_lo=24, n_hi=32, len_lo=16384,
             len_hi=32768),
        # long contexts under wide trees: the most arithmetic
        dict(name="tree_long_wide", op="tree", B=8, Hq=64, Hkv=8, D=128, dtype="f16", n_lo=64, n_hi=64, len_lo=16384,
             len_hi=32768),
        # acceptance: one tree, and a full batch of wide ones
        dict(name="accept_small", op="accept", B=1, n_lo=26, n_hi=26),
        dict(name="accept_batch", op="accept", B=256, n_lo=40, n_hi=64),
        # the accepted rows of one layer: one tree, and a full batch of the multi-head shape
        dict(name="commit_small", op="commit", B=1, Hkv=8, D=128, dtype="f16", n_lo=26, n_hi=26, len_lo=600,
             len_hi=600, take=5),
        dict(name="commit_batch", op="commit", B=256, Hkv=32, D=128, dtype="f16", n_lo=26, n_hi=64, len_lo=100,
             len_hi=900, take=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "tree", "accept", "commit"])
    most = [work(c) for c in listed()]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16, 32])
        Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 64])
        n_hi = _log(rng, 1, 128)
        n_lo = rng.randint(max(1, n_hi // 2), n_hi)
        len_hi = max(n_hi + 1, _log(rng, 1, 32768))
        len_lo = max(n_hi, rng.randint(1, len_hi))
        if op == "rope":
            c = dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                     dtype=rng.choice(["f16", "bf16"]), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(["none", "linear", "yarn"]), far=_log(rng, 64, 1 << 20))
        elif op == "tree":
            dtype = rng.choice(["f16", "bf16", "fp8"]) if D == 128 else rng.choice(["f16", "bf16"])
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, n_lo=n_lo, n_hi=n_hi,
                     len_lo=len_lo, len_hi=len_hi)
        elif op == "accept":
            c = dict(op=op, B=_log(rng, 1, 256), n_lo=n_lo, n_hi=n_hi)
        else:
            c = dict(op=op, B=_log(rng, 1, 256), Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]), n_lo=n_lo,
                     n_hi=n_hi, len_lo=len_lo, len_hi=min(len_hi, max(len_lo, 2048)), take=rng.randint(1, n_lo))
            if c["len_lo"] > c["len_hi"]:
                continue
        w = work(c)
        pool = c.get("B", 1) * c.get("len_hi", 1) * c.get("Hkv", 1) * c.get("D", 1) * 4
        scores = c.get("B", 1) * c.get("Hq", 1) * c.get("n_hi", 1) * c.get("len_hi", 1) * 4
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and pool <= 2 << 30 and scores <= 5 << 30:
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread: every seed has the same ones, in another order."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def work(case):
    c = case
    size = 1 if c.get("dtype") == "fp8" else 2
    if c["op"] == "rope":
        row = (2 * c["Hq"] + 4 * c["Hkv"]) * c["D"] * size + 16
        return {"bytes": c["T"] * row + c["rot"] * 4, "flops": c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    n = _spread(c["n_lo"], c["n_hi"], c["B"])
    if c["op"] == "accept":
        return {"bytes": int(n.sum()) * 20 + c["B"] * (4 * int(c["n_hi"]) + 16), "flops": int(n.sum())}
    if c["op"] == "commit":
        rows = int((_takes(c) - 1).sum())
        return {"bytes": rows * 4 * c["Hkv"] * c["D"] * size + c["B"] * (4 * c["take"] + 16), "flops": 0}
    L = _spread(c["len_lo"], c["len_hi"], c["B"])
    kv = int(L.sum()) * c["Hkv"] * (2 * c["D"] * size) + (int(L.sum()) * 8 if size == 1 else 0)
    words = -(-c["n_hi"] // 64)
    rows = int(n.sum())
    return {"bytes": kv + rows * (4 * c["Hq"] * c["D"] + 8 * words) + int(L.sum()) // 4,
            "flops": 4 * c["D"] * c["Hq"] * int((n * (L - n + 1)).sum())}


def _takes(c):
    """Nodes accepted per sequence of a commit case."""
    return _spread(1 if c["B"] > 1 else c["take"], c["take"], c["B"])


# ---- inputs ----------------------------------------------------------------
def _frequencies(rot, scaling):
    """Angle per position of each rotated pair, in 64 bits, and the factor on
    cosine and sine: base 10000; positions divided by 4; or, for a context 16
    times the trained one of 4096, the slow pairs divided by 16, the fast ones
    kept, and a ramp between 32 and 1 turns per trained context."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / 4.0, 1.0
    turned = lambda t: rot * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(turned(32.0)), 0), min(math.ceil(turned(1.0)), rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / 16.0 * ramp + f * (1.0 - ramp), 0.1 * math.log(16.0) + 1.0


def _forest(rng, n, n_hi):
    """Parents [B, n_hi] (-1: none) of random trees and the visibility of node
    j from node i [B, n_hi, n_hi]: itself and its ancestors."""
    B = len(n)
    parents = np.full((B, n_hi), -1, dtype=np.int32)
    sees = np.zeros((B, n_hi, n_hi), dtype=bool)
    rows = np.arange(B)
    for i in range(n_hi):
        if i:
            parents[:, i] = rng.integers(max(0, i - 6), i, size=B)
            sees[:, i] = sees[rows, parents[:, i]]
        sees[:, i, i] = True
    live = np.arange(n_hi)[None] < n[:, None]
    return np.where(live, parents, -1), sees & live[:, :, None] & live[:, None, :], live


def _words(sees, live):
    """Visibility as 64-bit words, the live nodes' rows packed: [T, words]."""
    B, n_hi, _ = sees.shape
    words = -(-n_hi // 64)
    bits = np.zeros((B, n_hi, words * 64), dtype=np.uint64)
    bits[:, :, :n_hi] = sees
    w = (bits.reshape(B, n_hi, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return w[live].view(np.int64)


def prepare(case, seed):
    c = case
    rng = np.random.Generator(np.random.PCG64(seed))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    randn = lambda shape, dt: torch.randn(shape, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    s = {"case": c}
    if c["op"] == "rope":
        T, H = c["T"], c["Hq"] + 2 * c["Hkv"]
        dt = KINDS[c["dtype"]]
        blocks = -(-T // BLOCK) + 3
        f, factor = _frequencies(c["rot"], c["scaling"])
        slots = rng.choice(blocks * BLOCK, size=T, replace=False)
        if T >= 16:
            slots[rng.choice(T, size=T // 16, replace=False)] = -1  # padded tokens
        # the projections' output, queries, keys and values of a token side by side
        qkv = randn((T, H * c["D"]), dt)
        q, k, v = qkv.split([c["Hq"] * c["D"], c["Hkv"] * c["D"], c["Hkv"] * c["D"]], dim=1)
        s |= {"q": q.unflatten(1, (c["Hq"], c["D"])), "k": k.unflatten(1, (c["Hkv"], c["D"])),
              "v": v.unflatten(1, (c["Hkv"], c["D"])), "positions": dev(rng.integers(0, c["far"], size=T)),
              "inv_freq": dev(f), "factor": factor, "slots": dev(slots.astype(np.int64)),
              "k_cache": randn((blocks, c["Hkv"], BLOCK, c["D"]), dt),
              "v_cache": randn((blocks, c["Hkv"], BLOCK, c["D"]), dt)}
        return s
    B = c["B"]
    n = rng.permutation(_spread(c["n_lo"], c["n_hi"], B))
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s["q_start"] = dev(q_start)
    if c["op"] != "commit":
        parents, sees, live = _forest(rng, n, c["n_hi"])
    if c["op"] == "accept":
        # drafts out of a small vocabulary, so that siblings may agree; after
        # most nodes the model picks one of the node's drafted children
        draft = rng.integers(0, 50, size=parents.shape)
        target = rng.integers(0, 50, size=parents.shape)
        rows = np.arange(B)
        for i in range(1, c["n_hi"]):
            hit = live[:, i] & (rng.random(B) < 0.7)
            target[rows[hit], parents[hit, i]] = draft[hit, i]
        s |= {"draft": dev(draft[live]), "target": dev(target[live]), "parents": dev(parents[live]),
              "max_path": c["n_hi"]}
        return s
    L = rng.permutation(_spread(c["len_lo"], c["len_hi"], B))
    nblk = -(-L // BLOCK)
    order = rng.permutation(int(nblk.sum()) + 3)
    tables = np.full((B, int(nblk.max())), -1, dtype=np.int32)
    tables[np.arange(tables.shape[1])[None] < nblk[:, None]] = order[:int(nblk.sum())]
    shape = (len(order), c["Hkv"], BLOCK, c["D"])
    s |= {"tables": dev(tables), "lens": dev(L.astype(np.int32)), "max_len": int(L.max()), "max_n": int(n.max())}
    if c["dtype"] == "fp8":
        code = lambda: (randn(shape, torch.float16) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
        scale = lambda: 0.005 + 0.01 * torch.rand((len(order), BLOCK), generator=gen, device="cuda")  # noqa: E731
        s |= {"k_cache": code(), "v_cache": code(), "k_scale": scale(), "v_scale": scale()}
    else:
        dt = KINDS[c["dtype"]]
        s |= {"k_cache": randn(shape, dt), "v_cache": randn(shape, dt), "k_scale": None, "v_scale": None}
    if c["op"] == "commit":
        take = np.minimum(rng.permutation(_takes(c)), n)
        path = np.full((B, c["take"]), -1, dtype=np.int32)
        for b in range(B):
            path[b, 1:take[b]] = 1 + np.sort(rng.choice(n[b] - 1, size=take[b] - 1, replace=False)) if take[b] > 1 else 0
            path[b, 0] = 0
        s |= {"path": dev(path), "path_len": dev(take.astype(np.int32))}
        return s
    s |= {"mask": dev(_words(sees, live)), "scale": 1.0 / math.sqrt(c["D"]),
          "q": randn((int(n.sum()), c["Hq"], c["D"]), KINDS.get(c["dtype"], torch.float16))}
    return s


# ---- one pass --------------------------------------------------------------
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_191_gb300 import ops
        if op == "rope":
            q = ops.rope_cache_write(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"],
                                     s["v_cache"], interleaved=s["case"]["interleaved"], factor=s["factor"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "tree":
            return ops.tree_attention(s["q"], s["q_start"], s["mask"], s["k_cache"], s["v_cache"], s["tables"],
                                      s["lens"], s["max_len"], s["max_n"], s["scale"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"])
        if op == "accept":
            path, count, token = ops.tree_accept(s["draft"], s["target"], s["parents"], s["q_start"], s["max_path"])
            return {"path": path, "path_len": count, "next_token": token}
        lens = ops.tree_commit(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["q_start"], s["path"],
                               s["path_len"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": lens}
    return {"rope": _rope, "tree": _tree, "accept": _accept, "commit": _commit}[op](s)


def _rope(s):
    c = s["case"]
    half = c["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]  # 64 bits: far positions turn many times
    cos, sin = ((t(angle) * s["factor"]).float()[:, None] for t in (torch.cos, torch.sin))

    def rotate(x):
        y = x.float()
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        u, w = a * cos - b * sin, a * sin + b * cos
        r = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    keep = s["slots"] >= 0
    blk, row = s["slots"][keep] // BLOCK, s["slots"][keep] % BLOCK
    s["k_cache"][blk, :, row] = rotate(s["k"])[keep]
    s["v_cache"][blk, :, row] = s["v"][keep]
    return {"q": rotate(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _paged(cache, scale, tables):
    """A cache's rows in each sequence's order, in 32 bits: [B, Hkv, tokens, D]."""
    at = tables.clamp(min=0).long()
    if scale is None:
        x = cache[at].float()
    else:
        x = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][:, :, None, :, None]
    return x.transpose(1, 2).flatten(2, 3)


def _tree(s):
    c = s["case"]
    T, Hq, D = s["q"].shape
    N, G = s["max_n"], Hq // c["Hkv"]
    start, count, L = s["q_start"][:-1].long(), s["q_start"].diff().long(), s["lens"].long()
    node = torch.arange(N, device=L.device)
    live = node[None] < count[:, None]
    at = (start[:, None] + node[None]).clamp(max=T - 1)
    K, V = _paged(s["k_cache"], s["k_scale"], s["tables"]), _paged(s["v_cache"], s["v_scale"], s["tables"])
    t = torch.arange(K.shape[2], device=L.device)
    # bit j of a node's words: whether it sees node j
    bits = (s["mask"][at][..., None] >> torch.arange(64, device=L.device) & 1).flatten(2).bool()
    j = (t[None] - (L - count)[:, None])  # node that key t is, < 0: context before the tree
    own_bit = torch.gather(bits, 2, j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, N, -1))
    sees = (j < 0)[:, None] | (own_bit & (j < count[:, None])[:, None])
    sees = sees & live[:, :, None] & (t[None] < L[:, None])[:, None]
    q = s["q"][at].float().unflatten(2, (c["Hkv"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, N G, D]
    x = (q @ K.transpose(2, 3)).unflatten(2, (N, G)) * s["scale"]
    x = x.masked_fill(~sees[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    V = V.masked_fill((t[None] >= L[:, None])[:, None, :, None], 0.0)
    out = (p.flatten(2, 3) @ V).unflatten(2, (N, G)) / total.clamp(min=1e-30)
    return out.permute(0, 2, 1, 3, 4).flatten(2, 3)[live].to(s["q"].dtype)


def _accept(s):
    start, count = s["q_start"][:-1].long(), s["q_start"].diff().long()
    T, B, N = s["draft"].numel(), start.numel(), s["max_path"]
    node = torch.arange(N, device=start.device)
    live = node[None] < count[:, None]
    at = (start[:, None] + node[None]).clamp(max=T - 1)
    parent = torch.where(live, s["parents"][at].long(), -1)
    draft, target = s["draft"][at], s["target"][at]
    hit = live & (parent >= 0) & (draft == torch.gather(target, 1, parent.clamp(min=0)))
    twin = (parent[:, :, None] == parent[:, None, :]) & hit[:, None, :] & (node[None, :] < node[:, None])
    hit = hit & ~twin.any(-1)  # the lowest of the children that agree
    # a node's ancestors by powers of "is the parent of": all of them have to be hit
    up = (parent[:, :, None] == node).float() + torch.eye(N, device=start.device)
    reach = torch.linalg.matrix_power(up, N) > 0
    taken = live & ((~reach) | (hit | (node == 0))[:, None]).all(-1)
    path_len = taken.sum(1)
    place = torch.where(taken, taken.cumsum(1) - 1, N)
    path = torch.full((B, N + 1), -1, dtype=torch.int64, device=start.device)
    path.scatter_(1, place, node.expand(B, -1))
    path[:, N] = -1
    last = torch.gather(path, 1, (path_len - 1).clamp(min=0)[:, None])
    token = torch.where(path_len > 0, torch.gather(target, 1, last.clamp(min=0))[:, 0], -1)
    return {"path": path[:, :N].int().contiguous(), "path_len": path_len.int(), "next_token": token}


def _commit(s):
    first = s["lens"].long() - s["q_start"].diff().long()  # position of node 0
    i = torch.arange(s["path"].shape[1], device=first.device)
    keep = i[None] < s["path_len"][:, None]
    b = torch.arange(first.numel(), device=first.device)[:, None].expand_as(keep)[keep]
    src, dst = (first[:, None] + s["path"].long())[keep], (first[:, None] + i[None])[keep]
    blk = lambda pos: s["tables"][b, pos // BLOCK].long()  # noqa: E731
    from_block, to_block = blk(src), blk(dst)
    rows = [s[x][from_block, :, src % BLOCK] for x in ("k_cache", "v_cache")]
    s["k_cache"][to_block, :, dst % BLOCK] = rows[0]
    s["v_cache"][to_block, :, dst % BLOCK] = rows[1]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": (first + s["path_len"]).int()}


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    """The computed numbers in 64 bits: rotation as a product of complex
    numbers, attention one sequence at a time.  Accepted paths and moved rows
    are not computed numbers."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        turn = s["factor"] * torch.exp(1j * (s["positions"].double()[:, None] * s["inv_freq"]))
        half = c["rot"] // 2

        def rotate(x):
            y = x.double().clone()
            if c["interleaved"]:
                z = torch.view_as_complex(y[..., :c["rot"]].unflatten(-1, (half, 2)).contiguous())
                y[..., :c["rot"]] = torch.view_as_real(z * turn[:, None]).flatten(-2)
            else:
                z = torch.complex(y[..., :half], y[..., half:c["rot"]]) * turn[:, None]
                y[..., :half], y[..., half:c["rot"]] = z.real, z.imag
            return y

        caches = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        slots = s["slots"][at]
        for name, x in (("k_cache", rotate(s["k"])), ("v_cache", s["v"].double())):
            flat = caches[name].transpose(1, 2).contiguous().flatten(0, 1)  # [slots, Hkv, D]
            flat[slots] = x[at]
            caches[name] = flat.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous()
        return {"q": rotate(s["q"]), **caches}
    if c["op"] != "tree":
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["q_start"].tolist(), s["lens"].tolist()
    words = s["mask"].cpu().numpy().view(np.uint64)
    G = c["Hq"] // c["Hkv"]
    for b, L in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        n = hi - lo
        at = s["tables"][b, :-(-L // BLOCK)].long()

        def rows(cache, scale):
            if scale is None:
                x = cache[at].double()
            else:
                x = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * scale[at].double()[:, None, :, None]
            return x.transpose(0, 1).flatten(1, 2)[:, :L]  # [Hkv, L, D]

        K, V = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
        sees = np.ones((n, L), dtype=bool)
        for i in range(n):
            for j in range(n):
                sees[i, L - n + j] = bool(int(words[lo + i, j // 64]) >> (j % 64) & 1)
        hidden = torch.from_numpy(~sees).cuda()
        for g in range(c["Hkv"]):
            x = torch.einsum("nhd,ld->hnl", s["q"][lo:hi, g * G:(g + 1) * G].double(), K[g]) * s["scale"]
            w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[lo:hi, g * G:(g + 1) * G] = torch.einsum("hnl,ld->nhd", w, V[g])
    return out
