"""GPU parity of the drafted-tree step (pa_rope_cache_write,
pa_tree_attention, pa_tree_accept, pa_tree_commit) against the float64
oracle, and the step as a whole.

Tolerances.  u is half a step of the 16-bit type the softmax weights are
rounded to (2^-11 f16, 2^-8 bf16), w the exact weights.
* Rounded weights, normalised by their own sum: every weight is off by at most
  u relative and the sum by as much, so the output by 2 u sum w |V|; f16
  weights below 2^-14 are off by 2^-25 of the largest instead, up to L of them.
* Scores: a float32 sum of D products is off by at most D 2^-23 sum |q K|
  scale, which moves a weight and the sum of weights by that much relative.
* 1-byte caches round weight x V scale instead of the weight: u once more.  In
  f16 a product below 2^-14 is off by 2^-25; weights are 2^4 at the reference,
  and so is their sum at least, and a product meets a code of at most 448:
  2^-29 x 448 for every key.
* 16-bit outputs: half a step.
Rotation: three float32 roundings and an angle within 2^-22: 2^-21 of |x1| +
|x2|, then half a step of the destination.
"""
import numpy as np
import pytest
import torch

from oracle import tree as O
from oracle.attention import paged_decode
from oracle.fp8_e4m3 import e4m3_decode
from paged_kv_cache_191_gb300 import ops, workloads as W
from tests.gpu_util import half_ulp, held_by_a_call_on_another_stream, np_exact, requires_cuda
from tests.tree_inputs import KV, TreeBatch, parents_of

pytestmark = [pytest.mark.gpu, requires_cuda]
DEV = "cuda"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def no_device_errors():
    ops.device_errors(clear=True)
    yield
    assert ops.device_errors(clear=True) == 0, "kernel flagged a device error"


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x
    return t.to(DEV) if dtype is None else t.to(DEV, dtype)


def args_of(w):
    """Positional and keyword arguments of ops.tree_attention."""
    sc = {} if w.k_scale is None else dict(k_scale=dev(w.k_scale), v_scale=dev(w.v_scale))
    return ([dev(w.q), dev(w.q_start), dev(w.mask), dev(w.k), dev(w.v), dev(w.tables), dev(w.lens),
             max(1, int(w.lens.max(initial=0))), max(1, int(w.sizes.max(initial=0))), w.scale], sc)


def run(w, out_dtype=torch.float32, **kw):
    a, sc = args_of(w)
    need = ops.tree_attention_workspace_size(w.Hq, a[8], a[3])
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN floats: stale scratch must not leak
    out = torch.full(w.q.shape, float("nan"), dtype=out_dtype, device=DEV)
    ops.tree_attention(*a, out=out, workspace=ws, **sc, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def oracle(w, k=None, v=None):
    return O.tree_attention(np_exact(w.q), w.q_start, w.mask, np_exact(w.k) if k is None else k,
                            np_exact(w.v) if v is None else v, w.tables, w.lens, w.scale,
                            None if w.k_scale is None else w.k_scale.numpy(),
                            None if w.v_scale is None else w.v_scale.numpy())


def check(out, w, ref=None, what=""):
    want, spread, score = ref or oracle(w)
    u = U[w.q.dtype]
    seen = np.repeat(w.lens.astype(np.float64), w.sizes)[:, None, None]
    tol = spread * ((2 if w.k_scale is None else 3) * u + 2 * w.D * 2.0 ** -23 * score[..., None] + 2.0 ** -18)
    if w.q.dtype == torch.float16:
        tol = tol + seen * 2.0 ** -25 * np.maximum(spread.max(-1, keepdims=True), 4.0)
        if w.k_scale is not None:
            tol = tol + seen * 2.0 ** -29 * 448
    if out.dtype != torch.float32:
        tol = tol + half_ulp(np.abs(want) + tol, out.dtype)
    got = out.double().numpy()
    assert np.isfinite(got).all(), what
    worst = (np.abs(got - want) / (tol + 1e-30)).max(initial=0.0)
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


SHAPES = [  # Hq, Hkv, D, cache, query
    (4, 4, 64, "f16", None), (8, 2, 128, "f16", None), (8, 1, 128, "bf16", None), (64, 8, 128, "bf16", None),
    (6, 2, 64, "bf16", None), (3, 1, 128, "f16", None), (24, 2, 128, "f16", None),
    (8, 2, 128, "fp8", torch.float16), (8, 2, 128, "fp8", torch.bfloat16), (16, 2, 128, "int8", torch.float16),
    (4, 2, 128, "int8", torch.bfloat16)]
BATCHES = [  # sizes, lengths
    ([1], [1]), ([5, 0, 33, 1], [5, 40, 300, 129]), ([64, 17, 65], [64, 128, 400]), ([16] * 7, [16, 17, 31, 127, 255, 256, 257]),
    ([150, 3], [700, 3])]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}{s[3]}-{str(s[4])[6:]}")
@pytest.mark.parametrize("bi", range(len(BATCHES)))
@pytest.mark.parametrize("masks", ["tree", "any"])
def test_ragged_batches(shape, bi, masks):
    Hq, Hkv, D, kind, qdt = shape
    w = TreeBatch(11 * bi + Hq, Hq, Hkv, D, kind, *BATCHES[bi], q_dtype=qdt, masks=masks)
    check(run(w), w, what=f"{shape} {BATCHES[bi]}")


@pytest.mark.parametrize("shape", [(8, 2, 128, "f16"), (16, 1, 128, "bf16"), (8, 8, 64, "f16"), (8, 1, 128, "int8")])
def test_items_that_span_many_ctas(shape):
    """Long contexts of few sequences: every item is cut over many CTAs, with
    boundaries inside and between items; 16-bit outputs."""
    w = TreeBatch(5, *shape, [9, 40, 2], [6000, 3001, 130])
    check(run(w, out_dtype=w.q.dtype), w)


@pytest.mark.parametrize("kind,D,odd", [("f16", 128, 0), ("f16", 128, 1), ("bf16", 64, 1), ("int8", 128, 0)])
def test_many_short_pieces_in_a_cta(kind, D, odd):
    """Items of one and two chunks, a dozen of them and more in every CTA, so that
    either warpgroup ends one while the other's next has begun: the same bits ten
    times over, and every row right."""
    B = 160
    rng = W.rng_for(40 + odd)
    lens = [int(x) for x in rng.integers(1, 129 if odd else 257, B)]
    w = TreeBatch(41, 16, 16, D, kind, [min(n, 1 + b % 9) for b, n in enumerate(lens)], lens)
    first = run(w)
    check(first, w)
    for _ in range(9):
        assert torch.equal(run(w), first)


@pytest.mark.parametrize("kind,sizes", [("f16", [40, 33, 0, 48]), ("int8", [40, 33, 48]), ("bf16", [100, 99])])
def test_items_side_by_side(kind, sizes):
    """Every sequence has the same number of items per kv head: 2 of 256 rows, 3
    of 128, 4; their CTAs go through the same chunks together."""
    w = TreeBatch(6, 16, 2, 128, kind, sizes, [3000, 1500, 700, 200][:len(sizes)])
    check(run(w), w)


@pytest.mark.parametrize("sizes", [[8, 8], [70, 70]])
def test_rows_that_see_nothing_are_zero(sizes):
    w = TreeBatch(21, 8, 2, 128, "f16", sizes, sizes)  # no context before the trees
    w.mask[:] = 0
    w.mask[3] = 1 << 2
    out = run(w)
    assert torch.count_nonzero(out[3]) > 0
    out[3] = 0
    assert torch.count_nonzero(out) == 0


def test_empty_context_and_more_nodes_than_context():
    w = TreeBatch(22, 8, 2, 128, "bf16", [4, 20, 150], [0, 12, 100], masks="any")
    out = run(w)
    assert ops.device_errors(clear=True) == ops.DEVERR_CONTEXT_LEN
    check(out, w)
    assert torch.count_nonzero(out[:4]) == 0


@pytest.mark.parametrize("kind", ["f16", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("G", [1, 24])
def test_unwritten_slots_reach_no_row(kind, G):
    """Pool rows that no token of the batch owns, and the rows of nodes no one
    sees, hold NaN (or, for 1-byte caches, NaN scales and codes)."""
    w = TreeBatch(23, 2 * G, 2, 128, kind, [12, 9, 20], [140, 40, 20], masks="any")
    dead = [(0, 5), (0, 11), (1, 0), (2, 7)]
    w.mask[:] |= 1 << 1
    for b, j in dead:
        w.mask[w.q_start[b]:w.q_start[b + 1]] &= ~(1 << j)
    ref = oracle(w)
    used = np.zeros(w.k.shape[:1] + (16,), dtype=bool)
    for b, L in enumerate(w.lens):
        t = np.arange(L)
        used[w.tables[b][t // 16], t % 16] = True
        for bb, j in dead:
            if bb == b:
                p = L - w.sizes[b] + j
                used[w.tables[b][p // 16], p % 16] = False
    at = torch.from_numpy(~used)
    for pool in (w.k, w.v):
        bad = torch.full((), float("nan")).to(pool.dtype) if kind in ("f16", "bf16") else torch.tensor(127, dtype=pool.dtype)
        pool.transpose(1, 2)[at] = bad
    if w.k_scale is not None:
        w.k_scale[at] = float("nan")
        w.v_scale[at] = float("nan")
    check(run(w), w, ref)


@pytest.mark.parametrize("kind,G", [("f16", 2), ("bf16", 40)])
def test_infinities_reach_the_rows_that_see_them_only(kind, G):
    w = TreeBatch(24, 2 * G, 2, 128, kind, [10, 6], [150, 30], masks="any")
    for b, j, val in ((0, 4, float("inf")), (0, 7, float("nan")), (1, 2, float("-inf"))):
        p = w.lens[b] - w.sizes[b] + j
        w.v[w.tables[b][p // 16], :, p % 16, 5] = val
    out = run(w).numpy()
    for b in range(2):
        for i in range(w.sizes[b]):
            row, bits = out[w.q_start[b] + i], O.visible(w.mask[w.q_start[b] + i], w.sizes[b])
            hit = bits[[4, 7]] if b == 0 else bits[[2]]
            if b == 0 and hit[1]:
                assert np.isnan(row[:, 5]).all()
            elif hit[0]:
                assert (row[:, 5] == (np.inf if b == 0 else -np.inf)).all()
            else:
                assert np.isfinite(row[:, 5]).all()
    fin = np.delete(out, 5, axis=2)
    for pool in (w.k, w.v):
        pool[~torch.isfinite(pool.float())] = 0
    want, spread, score = oracle(w)
    tol = np.delete(spread, 5, axis=2) * (2 * U[w.q.dtype] + 2.0 ** -15 * score[..., None] + 2.0 ** -18) + 1e-4
    assert (np.abs(fin - np.delete(want, 5, axis=2)) <= tol).all()


@pytest.mark.parametrize("kind,qdt", [("bf16", None), ("fp8", torch.float16), ("fp8", torch.bfloat16)])
@pytest.mark.parametrize("G", [1, 3, 16])
@pytest.mark.parametrize("before", [0, 20, 300])
def test_nan_values_reach_the_rows_that_see_them_only(kind, qdt, G, before):
    """Nodes with a NaN value in one dim, in the first chunk of a context and later:
    that dim of the rows that see them is NaN, all the rest is right."""
    w = TreeBatch(45, 2 * G, 2, 128, kind, [10, 6], [10 + before, 6 + before], q_dtype=qdt, masks="any")
    bad = [(0, 3), (0, 7), (1, 1)]
    at = [(w.tables[b][p // 16], p % 16) for b, j in bad for p in [w.lens[b] - w.sizes[b] + j]]
    for blk, row in at:
        w.v[blk, :, row, 77] = float("nan") if kind == "bf16" else 127  # (E4M3's NaN code)
    out = run(w)
    for blk, row in at:
        w.v[blk, :, row, 77] = 0
    hit = torch.tensor([any(b2 == b and O.visible(w.mask[w.q_start[b] + i], w.sizes[b])[j] for b2, j in bad)
                        for b in range(2) for i in range(w.sizes[b])])
    assert out[hit][..., 77].isnan().all() and 0 < hit.sum() < len(hit)
    want, spread, score = oracle(w)
    fix = hit[:, None] & (torch.arange(128) == 77)[None]
    got = torch.where(fix[:, None], torch.from_numpy(want), out.double()).numpy()
    tol = spread * (2 * U[w.q.dtype] + 2.0 ** -15 * score[..., None] + 2.0 ** -18) + 1e-6
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("scale", [-0.09, 0.0, 3.0])
def test_any_scale(scale):
    w = TreeBatch(25, 8, 2, 128, "f16", [9, 70], [200, 300])
    w.scale = scale
    check(run(w), w)


@pytest.mark.parametrize("kind", ["f16", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("G,sizes", [(2, [9, 20]), (8, [12, 16]), (16, [12, 20])])
def test_references_that_move(kind, G, sizes):
    """Scores that spread over tens of octaves, and grow along the context: 64
    rows of a kv head, 128, more."""
    w = TreeBatch(29, 2 * G, 2, 128, kind, sizes, [1500, 700])
    w.scale = 0.8
    if kind in ("f16", "bf16"):
        for b, L in enumerate(w.lens):
            for j, blk in enumerate(w.tables[b][:-(-L // 16)]):
                w.k[blk] = (w.k[blk].float() * (0.3 + 0.02 * j)).to(w.k.dtype)
    check(run(w), w)


@pytest.mark.parametrize("kind", ["f16", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("G", [2, 16, 48])
def test_a_nan_score_is_a_nan_row(kind, G):
    """Also where it is the only score; the rows that do not see it stay exact."""
    w = TreeBatch(30, 2 * G, 2, 128, kind, [6], [6])  # no context before the tree
    w.mask[:] = np.array([2, 4, 6, 0, 4, 2])[:, None]  # rows see nodes {1}, {2}, {1, 2}, {}, {2}, {1}
    blk = w.tables[0][0]
    if w.k_scale is None:
        v2 = np_exact(w.v)[blk, :, 2]
        w.k[blk, :, 1, 3] = float("nan")
    else:
        w.k_scale[blk, 1] = float("nan")
        dec = e4m3_decode if kind == "fp8" else (lambda c: c.view(np.int8).astype(np.float64))
        v2 = dec(w.v[blk, :, 2].numpy().view(np.uint8)) * float(w.v_scale[blk, 2])
    out = run(w).numpy()
    assert np.isnan(out[[0, 2, 5]]).all()
    assert (out[3] == 0).all()
    want = np.repeat(np.asarray(v2, dtype=np.float64), G, axis=0)  # a single key: its value
    tol = np.abs(want) * ((0 if w.k_scale is None else U[w.q.dtype]) + 2.0 ** -22)
    for i in (1, 4):
        assert (np.abs(out[i] - want) <= tol).all()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("G,sizes", [(2, [9, 20]), (8, [12, 16])])
def test_small_value_scales(kind, G, sizes):
    """Values of 2^-9 and of 2^6 of the usual size, next to one another."""
    w = TreeBatch(31, 2 * G, 2, 128, kind, sizes, [700, 90])
    w.v_scale *= 2.0 ** -9
    w.v_scale[::3] *= 2.0 ** 15
    check(run(w), w)
    w.v_scale[::3] *= 2.0 ** -15
    check(run(w), w)


def tight(w, small, what=""):
    """Relative to the row's own sums, with nothing for the size of the context but
    what 16-bit weights drop: float32 outputs within
    * spread u: one rounding of each weight (x V scale), whose sum, with 16-bit
      caches, is of the rounded weights: 2 u;
    * the scores' float32 sums (as above), 2^-18 for exponentials and references;
    * in f16, a weight below 2^-14 is off by 2^-25.  A row's largest weight (x V
      scale) is at least 2^small, so relative to it a key is off by 2^-25 - small, times
      the largest value (code) that can meet it, and all keys by `L` times that."""
    want, spread, score = oracle(w)
    most = O.tree_largest(np_exact(w.q), w.q_start, w.mask, np_exact(w.k), w.tables, w.lens, w.scale,
                          None if w.k_scale is None else w.k_scale.numpy(),
                          None if w.v_scale is None else w.v_scale.numpy())[..., None]
    u = U[w.q.dtype]
    tol = spread * ((2 if w.k_scale is None else 1) * u + 2 * w.D * 2.0 ** -23 * score[..., None] + 2.0 ** -18)
    top = {"fp8": 448.0, "int8": 127.0}.get(w.kind) or float(w.v.float().abs().max())
    if w.q.dtype == torch.float16:
        tol = tol + np.repeat(w.lens, w.sizes)[:, None, None] * 2.0 ** -(25 + small) * top * most
    # what the check is for: an output of zeros, or of half the size, does not pass
    assert (tol < 0.5 * np.abs(want)).mean() > 0.9, f"{what}: tolerance too wide to tell"
    got = run(w).double().numpy()
    assert np.isfinite(got).all(), what
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


@pytest.mark.parametrize("kind,qdt", [("fp8", torch.float16), ("int8", torch.float16), ("fp8", torch.bfloat16)])
@pytest.mark.parametrize("G,sizes", [(2, [9, 20]), (8, [12, 16])])
@pytest.mark.parametrize("octaves", [-40, -20, -9, 0, 12, 40])
def test_value_scales_of_any_size(kind, qdt, G, sizes, octaves):
    """V scales far below and above what f16 holds, all alike and next to usual ones."""
    w = TreeBatch(36, 2 * G, 2, 128, kind, sizes, [3000, 90], q_dtype=qdt)
    w.v_scale *= 2.0 ** octaves
    tight(w, 7, "alike")
    w.v_scale[::3] *= 2.0 ** -octaves
    tight(w, 7, "mixed")


@pytest.mark.parametrize("G", [2, 16])
def test_value_scales_of_zero_and_below(G):
    w = TreeBatch(37, 2 * G, 2, 128, "int8", [9, 12], [300, 40])
    w.v_scale[::3] *= -1
    w.v_scale[1::3] = 0
    want, spread, score = oracle(w)
    tol = spread * (U[torch.float16] + 2 * w.D * 2.0 ** -23 * score[..., None] + 2.0 ** -18)
    most = O.tree_largest(np_exact(w.q), w.q_start, w.mask, np_exact(w.k), w.tables, w.lens, w.scale, w.k_scale.numpy(),
                          w.v_scale.numpy())[..., None]
    tol = tol + 300 * 2.0 ** -32 * 127 * most
    assert (np.abs(run(w).double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("qdt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G", [1, 16])
def test_dominant_keys_with_value_scale_zero(kind, qdt, G):
    """Two of 140 octaves above the scores before them, in later chunks of a CTA, and
    one like them with a value: a third of it is the output."""
    w = TreeBatch(43, 64 * G, 64, 128, kind, [5, 5, 5], [600, 600, 600], q_dtype=qdt)
    exact_scores(w)
    w.scale = 1.0
    w.q[:] = 1
    w.k[:] = torch.where(torch.arange(128) % 3 > 0, 0x38 if kind == "fp8" else 1,
                         0xB8 if kind == "fp8" else -1).to(w.k.dtype)  # score 42
    for b in range(3):
        for at in (300, 430, 560):
            blk = w.tables[b][at // 16]
            w.k[blk, :, at % 16] = 0x38 if kind == "fp8" else 1  # score 128 x 1.1
            w.k_scale[blk, at % 16] = 1.1
            if at < 500:
                w.v_scale[blk, at % 16] = 0
    want, spread, _ = oracle(w)
    assert np.abs(want).max() > 1e-2
    got = run(w).double().numpy()
    assert (np.abs(got - want) <= spread * (U[qdt] + 2.0 ** -15) + 1e-30).all()


def exact_scores(w):
    """Queries and keys of -1, 0 and 1: products that float32 sums exactly, so that
    nothing but exponentials and the rounding of weights is off."""
    rng = W.rng_for(7)
    w.q = torch.from_numpy(rng.integers(-1, 2, w.q.shape)).to(w.q.dtype)
    k = torch.from_numpy(rng.integers(-1, 2, w.k.shape))
    if w.kind == "fp8":
        w.k = torch.where(k == 0, 0, torch.where(k > 0, 0x38, 0xB8)).to(torch.uint8)
    else:
        w.k = k.to(w.k.dtype)
    if w.k_scale is not None:
        w.k_scale[:] = 1
    w.scale = 0.25


def check_weights(w, u):
    """Float32 outputs, weights of half a step u: the scores in octaves are below 64 (at
    a scale of 0.25), off by 2^-24 of that (a weight by 2^-18), exponentials by 2^-22; a
    part's reference and the merge as much again: 2^-17.  f16 products are at least 2^7 at a row's
    largest (as above).  The product's float32 sum goes on 16 keys at a time, 2^-23 each."""
    want, spread, _ = oracle(w)
    steps = np.repeat(-(-w.lens // 16), w.sizes)[:, None, None]
    tol = spread * (u + 2.0 ** -17 * max(1.0, w.scale / 0.25) + steps * 2.0 ** -23)
    if w.k_scale is not None and w.q.dtype == torch.float16:
        most = O.tree_largest(np_exact(w.q), w.q_start, w.mask, np_exact(w.k), w.tables, w.lens, w.scale,
                              w.k_scale.numpy(), w.v_scale.numpy())[..., None]
        tol = tol + np.repeat(w.lens, w.sizes)[:, None, None] * 2.0 ** -32 * {"fp8": 448, "int8": 127}[w.kind] * most
    worst = (np.abs(run(w).double().numpy() - want) / (tol + 1e-30)).max()  # (rows that see nothing are 0)
    assert worst <= 1.0, f"{worst:.2f} of the tolerance"


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("qdt,u", [(torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -16)])
@pytest.mark.parametrize("G,sizes", [(1, [9, 0, 3]), (2, [9, 20, 3]), (8, [12, 16, 3])])
@pytest.mark.parametrize("scale", [0.25, 4.0])
def test_weights_over_one_byte_caches(kind, qdt, u, G, sizes, scale):
    """11 bits with f16 queries; with bf16 ones 16 bits, down to the smallest weights."""
    w = TreeBatch(38, 2 * G, 2, 128, kind, sizes, [700, 40, 3], q_dtype=qdt, masks="any")
    exact_scores(w)
    w.scale = scale
    check_weights(w, u)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,sizes", [(1, [9, 0, 3]), (2, [9, 16, 3]), (3, [12, 4, 1]), (8, [12, 16, 3]), (16, [30, 16, 3])])
@pytest.mark.parametrize("masks", ["tree", "any"])
def test_weights_over_bf16_caches_have_16_bits(D, G, sizes, masks):
    """Their sum of two bf16 is off by a half step of a half step, 2^-16; so is the
    sum that divides, where it is of the rounded weights."""
    w = TreeBatch(39, 2 * G, 2, D, "bf16", sizes, [700, 40, 3], masks=masks)
    exact_scores(w)
    check_weights(w, 2.0 ** -15)


@pytest.mark.parametrize("G", [1, 2, 8])
def test_a_bf16_chain_is_as_exact_as_chunked_prefill(G):
    """The same causal rows through both calls, float32 outputs."""
    w = TreeBatch(40, 2 * G, 2, 128, "bf16", [16, 9], [900, 70])
    exact_scores(w)
    for b, n in enumerate(w.sizes):
        for i in range(n):
            w.mask[w.q_start[b] + i] = (1 << (i + 1)) - 1
    a, _ = args_of(w)
    want, spread, _ = oracle(w)
    chunks = ops.chunked_prefill(a[0], a[1], a[3], a[4], a[5], a[6], a[7], a[8], a[9], out_dtype=torch.float32)
    for out in (chunks.cpu(), run(w)):
        assert (np.abs(out.double().numpy() - want) <= spread * 2.0 ** -14).all()


@pytest.mark.parametrize("G", [2, 16])
def test_small_weights_beside_large_ones(G):
    """In every 128 keys one with value 0; the others, of e^-16 of its weight, which f16
    would round 6 % off, are the whole output."""
    w = TreeBatch(42, 2 * G, 2, 128, "f16", [5], [3000])
    one = torch.where(torch.arange(128) % 3 == 0, 1.0, -1.0).half()
    i = torch.arange(128)
    w.q[:], w.k[:] = one, one * torch.where(i < 64, 1.0, -1.0).half()
    w.scale = 0.25
    w.v = w.v.abs()
    blk = torch.from_numpy(w.tables[0][2:-1:8].astype(np.int64))
    w.k[blk, :, 5] = one * torch.where(i < 96, 1.0, -1.0).half()  # score 64 x 0.25, the others' 0
    w.v[blk, :, 5] = 0
    tight(w, 7)


def test_a_chain_is_chunked_prefill():
    w = TreeBatch(26, 16, 4, 128, "bf16", [40, 3, 17], [900, 3, 64])
    for b, n in enumerate(w.sizes):
        for i in range(n):
            w.mask[w.q_start[b] + i] = (1 << (i + 1)) - 1
    a, _ = args_of(w)
    want = ops.chunked_prefill(a[0], a[1], a[3], a[4], a[5], a[6], a[7], a[8], a[9], out_dtype=torch.float32)
    check(run(w), w)
    check(want.cpu(), w)


def test_the_same_bits_again_and_for_other_blocks():
    w = TreeBatch(27, 16, 2, 128, "f16", [30, 9], [2000, 800])
    one, two = run(w, out_dtype=torch.float16), run(w, out_dtype=torch.float16)
    perm = torch.from_numpy(W.rng_for(1).permutation(w.k.shape[0]))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm))
    w.k, w.v = w.k[perm].contiguous(), w.v[perm].contiguous()
    w.tables = np.where(w.tables >= 0, inv.numpy()[np.maximum(w.tables, 0)], -1).astype(np.int32)
    assert torch.equal(one, two) and torch.equal(one, run(w, out_dtype=torch.float16))


def test_rows_of_no_sequence_and_long_sequences_are_left_alone():
    w = TreeBatch(28, 8, 2, 128, "f16", [6, 30, 5], [50, 90, 70])
    a, _ = args_of(w)
    ref = oracle(w)
    q = torch.cat([a[0], torch.randn_like(a[0][:7])])
    mask = torch.cat([a[2], a[2][:7]])
    out = torch.full(q.shape, 7.0, dtype=torch.float32, device=DEV)
    ops.tree_attention(q, a[1], mask, *a[3:8], 8, w.scale, out=out)  # sequence 1 has 30 > 8 nodes
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE
    out = out.cpu()
    assert (out[6:36] == 7).all() and (out[41:] == 7).all()
    keep = np.r_[0:6, 36:41]
    assert np.abs(out.numpy()[keep] - ref[0][keep]).max() < 1e-2


def test_bad_blocks_are_flagged():
    w = TreeBatch(29, 8, 2, 128, "f16", [6], [200])
    w.tables[0, 2] = w.k.shape[0] + 9
    run(w)
    assert ops.device_errors(clear=True) == ops.DEVERR_BLOCK_RANGE
    w.tables[0, 2] = -5
    run(w)
    assert ops.device_errors(clear=True) == ops.DEVERR_BLOCK_RANGE


def test_graph_replays_follow_the_inputs():
    """Two captured calls with a workspace each, replayed on two streams after
    their inputs changed; lengths, tables and trees are read at replay."""
    ws = [TreeBatch(s, 8, 2, 128, "f16", [12, 5], [L, 400]) for s, L in ((31, 1500), (32, 700))]
    nxt = [TreeBatch(s, 8, 2, 128, "f16", [3, 14], [90, 390]) for s in (33, 34)]
    calls = []
    for w in ws:
        a, _ = args_of(w)
        a[5] = torch.full((2, 100), -1, dtype=torch.int32, device=DEV)
        a[5][:, :w.tables.shape[1]] = dev(w.tables)
        a[7], a[8] = 1600, 20
        scratch = torch.empty(ops.tree_attention_workspace_size(8, 20, a[3]), dtype=torch.uint8, device=DEV)
        out = torch.empty(17, 8, 128, dtype=torch.float32, device=DEV)
        ops.tree_attention(*a, out=out, workspace=scratch)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.tree_attention(*a, out=out, workspace=scratch)
        calls.append((g, a, out, scratch))  # a captured call's buffers have to stay alive
    for batch in (ws, nxt, ws):
        for (g, a, out, _), w in zip(calls, batch):
            a[0].copy_(w.q)
            a[1].copy_(torch.from_numpy(w.q_start))
            a[2].copy_(torch.from_numpy(w.mask))
            for t, src in ((a[3], w.k), (a[4], w.v)):
                t[:min(len(t), len(src))].copy_(src[:min(len(t), len(src))])
            a[5].fill_(-1)
            a[5][:, :w.tables.shape[1]] = dev(w.tables)
            a[6].copy_(torch.from_numpy(w.lens))
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (g, *_), s in zip(calls, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, out, _), w in zip(calls, batch):
            check(out.cpu(), w)


@pytest.mark.parametrize("what", ["rope", "attention", "accept", "commit"])
def test_a_call_keeps_its_memory_on_another_stream(monkeypatch, what):
    w = TreeBatch(35, 8, 2, 128, "f16", [12, 5], [1500, 400])
    a, _ = args_of(w)
    f, _ = ops.rope_frequencies(64, device=DEV)
    k = torch.randn(17, 2, 128, device=DEV).half()
    no_slot, pos = torch.full((17,), -1, device=DEV), torch.arange(17, device=DEV)
    par = dev(np.concatenate(w.parents))
    tok = torch.zeros(17, dtype=torch.int64, device=DEV)
    path, n = dev(np.zeros((2, 1), np.int32)), dev(np.ones(2, np.int32))
    call = {"rope": lambda s: [ops.rope_cache_write(a[0], k, k, pos, f, no_slot, a[3], a[4], stream=s)],
            "attention": lambda s: [ops.tree_attention(*a, stream=s)],
            "accept": lambda s: list(ops.tree_accept(tok, tok, par, a[1], 12, stream=s)),
            "commit": lambda s: [ops.tree_commit(*a[3:7], a[1], path, n, stream=s)]}[what]
    plain, other = held_by_a_call_on_another_stream(monkeypatch, ops, call)
    assert all(torch.equal(x, y) for x, y in zip(plain, other))


# ---- rotary cache write --------------------------------------------------------
def rope_case(seed, T, Hq, Hkv, D, dt, kind, rot, far=4096):
    rng = W.rng_for(seed)
    blocks = -(-T // 16) + 4
    slots = rng.choice(blocks * 16, size=T, replace=False).astype(np.int64)
    if T > 3:
        slots[rng.choice(T, size=max(1, T // 5), replace=False)] = -1
    pos = rng.integers(0, far, T)
    qkv = W.randn(rng, (T, Hq + 2 * Hkv, D), dt).to(DEV)
    if kind in ("fp8", "int8"):
        kc = torch.full((blocks, Hkv, 16, D), 3, dtype=KV[kind], device=DEV)
        sc = [torch.full((blocks, 16), 5.0, device=DEV) for _ in range(2)]
    else:
        kc, sc = W.randn(rng, (blocks, Hkv, 16, D), KV[kind]).to(DEV), [None, None]
    return qkv, slots, pos, kc, kc.clone(), sc


def step16(x, dtype):
    return half_ulp(x, dtype) if dtype != torch.float32 else 0.0


@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 4, 4, 64, 64), (5, 8, 2, 128, 128), (37, 3, 1, 128, 32),
                                            (700, 8, 4, 128, 64), (9, 0, 2, 64, 16), (350, 64, 32, 128, 128)])
@pytest.mark.parametrize("dt,kind", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f16"), ("f32", "bf16"), ("f16", "fp8"),
                                     ("bf16", "int8"), ("f32", "fp8"), ("f32", "int8")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_write(T, Hq, Hkv, D, rot, dt, kind, interleaved):
    if kind in ("fp8", "int8") and D != 128:
        pytest.skip("1-byte caches have head_dim 128")
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dt]
    qkv, slots, pos, kc, vc, (ks, vs) = rope_case(T + D, T, Hq, Hkv, D, dtype, kind, rot)
    k0, v0 = kc.clone(), vc.clone()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f, _ = ops.rope_frequencies(rot, device=DEV)
    got = ops.rope_cache_write(q if Hq else None, k, v, dev(pos), f, dev(slots), kc, vc, interleaved, 1.25,
                               k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    if Hq:
        want, mag = O.rotate(np_exact(q), pos, f.cpu().numpy(), 1.25, interleaved)
        tol = mag * 2.0 ** -21 + step16(np.abs(want) + mag * 2.0 ** -21, dtype)
        assert got.dtype == dtype and (np.abs(got.cpu().double().numpy() - want) <= tol).all()
    else:
        assert got is None
    keep = np.nonzero(slots >= 0)[0]
    blk, row = slots[keep] // 16, slots[keep] % 16
    untouched = np.ones((kc.shape[0], 16), dtype=bool)
    untouched[blk, row] = False
    for cache, old, src, sc, rotated in ((kc, k0, k, ks, True), (vc, v0, v, vs, False)):
        x = np_exact(src)
        want, mag = O.rotate(x, pos, f.cpu().numpy(), 1.25, interleaved) if rotated else (x.astype(np.float64), abs(x))
        want, mag = want[keep], mag[keep] * (2.0 ** -21 if rotated else 0.0)
        rows = np_exact(cache).transpose(0, 2, 1, 3)[blk, row]
        if sc is None:
            tol = mag + (step16(np.abs(want) + mag, cache.dtype) if rotated or dtype != cache.dtype else 0.0)
            assert (np.abs(rows.astype(np.float64) - want) <= tol).all()
        else:
            scale = sc.cpu().numpy()[blk, row].astype(np.float64)[:, None, None]
            amax = np.abs(want).max(axis=(1, 2), keepdims=True)
            off = mag.max(axis=(1, 2), keepdims=True)
            top = 127.0 if kind == "int8" else 448.0
            assert (np.abs(scale - amax / top) <= (off + amax * 2.0 ** -23) / top).all()
            val = (rows.astype(np.float64) if kind == "int8" else e4m3_decode(rows)) * scale
            step = 0.5 * scale if kind == "int8" else np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10)
            assert (np.abs(val - want) <= step * (1 + 2.0 ** -10) + 2 * off + amax * 2.0 ** -20).all()
        at = torch.from_numpy(untouched)
        assert torch.equal(cache.cpu().transpose(1, 2)[at], old.cpu().transpose(1, 2)[at])
        if sc is not None:
            assert (sc.cpu()[at] == 5).all()


def test_rope_far_and_negative_positions():
    pos = np.array([0, 1, -1, 2 ** 20, 2 ** 31 + 7, -(2 ** 40), 2 ** 50 + 3], dtype=np.int64)
    qkv, _, _, kc, vc, _ = rope_case(3, 7, 2, 1, 128, torch.float32, "f16", 128)
    f, _ = ops.rope_frequencies(128, device=DEV)
    got = ops.rope_cache_write(qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], dev(pos), f, dev(np.full(7, -1)), kc, vc)
    want, mag = O.rotate(np_exact(qkv[:, :2]), pos, f.cpu().numpy())
    # the frequency in turns is known to 2^-53, so the angle to |pos| 2^-52 radians and a bit
    tol = mag * (2.0 ** -21 + np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -51)
    assert (np.abs(got.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rope_frequency_that_is_no_number(bad):
    """Its pair becomes NaN, the others stay."""
    qkv, slots, pos, kc, vc, _ = rope_case(11, 9, 2, 1, 64, torch.float32, "f16", 64)
    f, _ = ops.rope_frequencies(64, device=DEV)
    call = lambda f: ops.rope_cache_write(qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], dev(pos), f, dev(slots), kc, vc)  # noqa: E731
    want = call(f)
    f[5] = bad
    got = call(f)
    pair = torch.tensor([5, 37], device=DEV)
    assert got[..., pair].isnan().all()
    rest = torch.ones(64, dtype=torch.bool, device=DEV)
    rest[pair] = False
    assert torch.equal(got[..., rest], want[..., rest])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_in_a_packed_projection(interleaved):
    qkv, slots, pos, kc, vc, _ = rope_case(8, 40, 8, 2, 128, torch.bfloat16, "bf16", 64)
    f, a = ops.rope_frequencies(64, scaling="yarn", factor=16.0, device=DEV)
    plain = [t.contiguous() for t in (qkv[:, :8], qkv[:, 8:10], qkv[:, 10:])]
    k2, v2, before = kc.clone(), vc.clone(), qkv.clone()
    want = ops.rope_cache_write(*plain, dev(pos), f, dev(slots), k2, v2, interleaved, a)
    got = ops.rope_cache_write(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], dev(pos), f, dev(slots), kc, vc, interleaved, a,
                               q_out=qkv[:, :8])
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want)
    assert torch.equal(kc, k2) and torch.equal(vc, v2) and torch.equal(qkv[:, 8:], before[:, 8:])


def test_rope_slot_past_the_pool_and_no_tokens():
    qkv, slots, pos, kc, vc, _ = rope_case(9, 6, 4, 2, 128, torch.float16, "f16", 128)
    f, _ = ops.rope_frequencies(128, device=DEV)
    slots[2] = kc.shape[0] * 16
    slots[4] = -1
    k0 = kc.clone()
    got = ops.rope_cache_write(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], dev(pos), f, dev(slots), kc, vc)
    assert ops.device_errors(clear=True) == ops.DEVERR_SLOT_RANGE
    want, mag = O.rotate(np_exact(qkv[:, :4]), pos, f.cpu().numpy())
    assert (np.abs(got.cpu().double().numpy() - want) <= mag * 2.0 ** -21 + half_ulp(np.abs(want) + 1e-6, torch.float16)).all()
    changed = (kc != k0).any(-1).any(1).sum().item()
    assert changed == (slots >= 0).sum() - 1
    e = ops.rope_cache_write(qkv[:0, :4], qkv[:0, 4:6], qkv[:0, 6:], dev(pos[:0]), f, dev(slots[:0]), kc, vc)
    assert e.shape == (0, 4, 128)


def test_calls_refuse_wrong_tensors():
    qkv, slots, pos, kc, vc, _ = rope_case(10, 6, 4, 2, 128, torch.float16, "f16", 128)
    f, _ = ops.rope_frequencies(128, device=DEV)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    good = [q, k, v, dev(pos), f, dev(slots), kc, vc]
    for i, bad in ((0, q.transpose(1, 2)), (1, k[:, :1]), (2, v.float()), (3, dev(pos).int()), (4, f.float()),
                   (5, dev(slots)[:5]), (7, vc[:2]), (6, kc.transpose(0, 1))):
        a = list(good)
        a[i] = bad
        with pytest.raises((ValueError, ops.PagedKVError)):
            ops.rope_cache_write(*a)
    w = TreeBatch(12, 8, 2, 128, "f16", [5, 4], [40, 30])
    good, _ = args_of(w)
    for i, bad in ((0, good[0][:, :, ::2]), (1, good[1].long()), (2, good[2].int()), (2, good[2][:4]),
                   (4, good[4][:1]), (5, good[5][:1]), (6, good[6].long()), (8, 65)):
        a = list(good)
        a[i] = bad
        with pytest.raises((ValueError, ops.PagedKVError)):
            ops.tree_attention(*a)
    with pytest.raises(ops.PagedKVError):
        ops.tree_attention(*good, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ops.PagedKVError):
        ops.tree_attention(*good, k_scale=torch.ones(w.k.shape[0], 16, device=DEV),
                           v_scale=torch.ones(w.k.shape[0], 16, device=DEV))


# ---- acceptance and commit ---------------------------------------------------------
def accept_case(seed, sizes, vocab=4):
    rng = W.rng_for(seed)
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    par = np.concatenate([parents_of(rng, n) for n in sizes] + [np.zeros(0, np.int32)])
    draft, target = (rng.integers(0, vocab, qs[-1]) for _ in range(2))
    return qs, par, draft, target


@pytest.mark.parametrize("sizes,max_path", [([1], 1), ([26], 26), ([0, 7, 64, 1, 130], 64), ([40] * 300, 9),
                                            ([3000, 5], 3000), ([2048, 2049], 4)])
def test_accept(sizes, max_path):
    qs, par, draft, target = accept_case(len(sizes) + max_path, sizes, vocab=2)
    path, n, tok = ops.tree_accept(dev(draft), dev(target), dev(par), dev(qs), max_path)
    want, want_tok = O.tree_accept(draft, target, par, qs, max_path)
    assert n.tolist() == [len(p) for p in want] and tok.tolist() == want_tok
    assert path.tolist() == [p + [-1] * (max_path - len(p)) for p in want]


def test_accept_malformed_parents():
    par = np.array([5, 0, 3, 1, -7, -1, 1], dtype=np.int32)  # node 0's is not read; 2 -> 3 and -7 are malformed
    same = np.zeros(7, dtype=np.int64)
    path, n, _ = ops.tree_accept(dev(same), dev(same), dev(par), dev(np.array([0, 7], np.int32)), 7)
    assert ops.device_errors(clear=True) == ops.DEVERR_TREE
    assert path[0].tolist() == [0, 1, 3, -1, -1, -1, -1] and n.tolist() == [3]
    path, n, tok = ops.tree_accept(dev(same), dev(same), dev(par), dev(np.array([0, 9, 3], np.int32)), 4)
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE
    assert n.tolist() == [0, 0] and tok.tolist() == [-1, -1] and (path == -1).all()


@pytest.mark.parametrize("kind,Hkv,D", [("f16", 2, 64), ("bf16", 8, 128), ("fp8", 3, 128), ("int8", 32, 128)])
@pytest.mark.parametrize("sizes,lens", [([1], [1]), ([26, 0, 7, 64], [26, 9, 100, 333]), ([600], [700])])
def test_commit(kind, Hkv, D, sizes, lens):
    w = TreeBatch(D + Hkv, Hkv, Hkv, D, kind, sizes, lens)
    rng = W.rng_for(2)
    paths = []
    for n in sizes:
        m = int(rng.integers(1, n + 1)) if n else 0
        m = n - 5 if n == 600 else m  # more moves than are staged at a time
        paths.append([0] + sorted(int(x) for x in 1 + rng.choice(n - 1, m - 1, replace=False)) if m else [])
    wide = max(sizes)
    path = np.full((len(sizes), wide), -1, dtype=np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    caches = [w.k, w.v] + ([w.k_scale, w.v_scale] if w.k_scale is not None else [])
    on = [c.to(DEV) for c in caches]
    lens_out = ops.tree_commit(on[0], on[1], dev(w.tables), dev(w.lens), dev(w.q_start), dev(path),
                               dev(np.array([len(p) for p in paths], np.int32)), *(on[2:] or [None, None]))
    want, want_lens = O.tree_commit([np_exact(c) for c in caches], w.tables, w.lens, w.q_start, paths)
    assert lens_out.tolist() == want_lens
    for c, x in zip(on, want):
        assert np.array_equal(np_exact(c), x)


@pytest.mark.parametrize("path,n,flag", [([0, 0, 2], 3, "TREE"), ([0, 3, 2], 3, "TREE"), ([1, 1, 2], 2, "TREE"),
                                         ([0, 2, 9], 3, "TREE"), ([0, 2, 4], -1, "TREE"), ([0, 2, 4], 4, "TREE")])
def test_commit_moves_nothing_for_a_bad_path(path, n, flag):
    w = TreeBatch(6, 4, 4, 128, "f16", [6, 6], [40, 40])
    k, v = w.k.to(DEV), w.v.to(DEV)
    p = np.array([path, [0, 2, 5]], dtype=np.int32)
    lens = ops.tree_commit(k, v, dev(w.tables), dev(w.lens), dev(w.q_start), dev(p), dev(np.array([n, 3], np.int32)))
    assert ops.device_errors(clear=True) == getattr(ops, "DEVERR_" + flag)
    want, _ = O.tree_commit([w.k.numpy()], w.tables, w.lens, w.q_start, [[], [0, 2, 5]])
    assert lens.tolist() == [40, 37] and np.array_equal(np_exact(k), want[0])


def test_commit_flags_lengths_and_blocks():
    w = TreeBatch(7, 4, 4, 128, "f16", [6, 6, 6], [40, 4, 40])
    w.tables[2, 2] = 1000
    k, v = w.k.to(DEV), w.v.to(DEV)
    path = np.array([[0, 2]] * 3, np.int32)
    lens = ops.tree_commit(k, v, dev(w.tables), dev(w.lens), dev(w.q_start), dev(path), dev(np.array([2] * 3, np.int32)))
    assert ops.device_errors(clear=True) == ops.DEVERR_CONTEXT_LEN | ops.DEVERR_BLOCK_RANGE
    assert lens.tolist() == [36, 4, 40]


# ---- the step as a whole -------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f16", "bf16", "fp8", "int8"])
def test_a_speculative_step(kind):
    """Allocate, append the trees, rotate and write, attend, accept, commit and
    truncate, three steps over; the caches then hold what writing the accepted
    tokens alone gives, and a decode over them agrees with the oracle.  All on
    another stream than the default one."""
    rng = W.rng_for(77)
    Hq, Hkv, D, B = 8, 2, 128, 3
    dt = KV[kind] if kind in ("f16", "bf16") else torch.float16
    blocks = 64
    shape = (blocks, Hkv, 16, D)
    quant = kind in ("fp8", "int8")
    kc, vc = (torch.zeros(shape, dtype=KV[kind], device=DEV) for _ in range(2))
    k2, v2 = kc.clone(), vc.clone()
    sc = [torch.ones(blocks, 16, device=DEV) for _ in range(4)] if quant else [None] * 4
    alloc, plain = ops.BlockAllocator(blocks), ops.BlockAllocator(blocks)
    f, factor = ops.rope_frequencies(64, device=DEV)
    ids, prompt = list(range(B)), [37, 5, 80]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for b in ids:  # prompts, written the same way to both pools
            for a, (k, v), (ks, vs) in ((alloc, (kc, vc), sc[:2]), (plain, (k2, v2), sc[2:])):
                a.alloc_seq(b, 0)
                slots, _ = a.append_tokens(b, prompt[b])
                g = W.rng_for(b)
                x = [W.randn(g, (prompt[b], Hkv, D), dt).to(DEV) for _ in range(2)]
                ops.rope_cache_write(None, x[0], x[1], torch.arange(prompt[b], device=DEV), f,
                                     torch.tensor(slots, device=DEV), k, v, factor=factor, k_scale=ks, v_scale=vs)
        for _ in range(3):
            sizes = [int(rng.integers(1, 30)) for _ in ids]
            before = [alloc.table(b)[1] for b in ids]
            qs, par, draft, target = accept_case(int(rng.integers(1 << 30)), sizes, vocab=2)
            mask, depth = ops.tree_mask(par, qs)
            pos = np.concatenate([before[b] + depth[qs[b]:qs[b + 1]] for b in ids]).astype(np.int64)
            slots = sum((alloc.append_tokens(b, n)[0] for b, n in zip(ids, sizes)), [])
            tables, lens = alloc.tables(ids, 24)
            T = int(qs[-1])
            q, k, v = (W.randn(rng, (T, h, D), dt).to(DEV) for h in (Hq, Hkv, Hkv))
            q = ops.rope_cache_write(q, k, v, dev(pos), f, torch.tensor(slots, device=DEV), kc, vc, factor=factor,
                                     k_scale=sc[0], v_scale=sc[1])
            tb, ln, st = dev(tables), dev(lens), dev(qs)
            out = ops.tree_attention(q, st, dev(mask), kc, vc, tb, ln, int(lens.max()), max(sizes), D ** -0.5,
                                     out_dtype=torch.float32, k_scale=sc[0], v_scale=sc[1])
            s.synchronize()
            w = TreeBatch.__new__(TreeBatch)
            w.q, w.q_start, w.mask, w.k, w.v, w.tables, w.lens = q.cpu(), qs, mask, kc.cpu(), vc.cpu(), tables, lens
            w.k_scale, w.v_scale = (x.cpu() if quant else None for x in sc[:2])
            w.scale, w.D, w.sizes = D ** -0.5, D, np.array(sizes)
            check(out.cpu(), w)
            path, n, _ = ops.tree_accept(dev(draft), dev(target), dev(par), st, 8)
            new = ops.tree_commit(kc, vc, tb, ln, st, path, n, sc[0], sc[1]).tolist()
            paths = [p[:m] for p, m in zip(path.tolist(), n.tolist())]
            for b in ids:
                assert new[b] == before[b] + len(paths[b])
                alloc.truncate_seq(b, new[b])
                # the accepted tokens alone, one after the other, in the other pool
                at = [int(qs[b]) + i for i in paths[b]]
                slots, _ = plain.append_tokens(b, len(at))
                ops.rope_cache_write(None, k[at], v[at], torch.arange(before[b], new[b], device=DEV), f,
                                     torch.tensor(slots, device=DEV), k2, v2, factor=factor, k_scale=sc[2],
                                     v_scale=sc[3])
        s.synchronize()
        for b in ids:
            ta, n1 = alloc.table(b)
            tp, n2 = plain.table(b)
            assert n1 == n2
            t = np.arange(n1)
            ia, ip = (torch.from_numpy(np.array(x)[t // 16] * 16 + t % 16).to(DEV) for x in (ta, tp))
            for x, y in ((kc, k2), (vc, v2)):
                flat = lambda c: c.transpose(1, 2).reshape(-1, Hkv, D).view(torch.uint8)  # noqa: E731
                assert torch.equal(flat(x)[ia], flat(y)[ip])
            for x, y in zip(sc[:2], sc[2:]):
                assert x is None or torch.equal(x.reshape(-1)[ia], y.reshape(-1)[ip])
        tables, lens = alloc.tables(ids, 24)
        q = W.randn(rng, (B, Hq, D), dt).to(DEV)
        out = ops.decode(q, kc, vc, dev(tables), dev(lens), int(lens.max()), D ** -0.5, out_dtype=torch.float32,
                         k_scale=sc[0], v_scale=sc[1])
        s.synchronize()
    cp = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    ref = paged_decode(np_exact(q), np_exact(kc), np_exact(vc), tables, lens, D ** -0.5, cp(sc[0]), cp(sc[1]))
    assert np.abs(out.cpu().numpy() - ref).max() < (2e-2 if quant else 2e-3)
