"""GPU parity of the block-scaled cache (pa_block_scaled_append, _attention,
_copy) and of pa_draft_verify against the float64 oracle, and a speculative
step of them together.

Codes, scales, paths and drawn tokens are equal to the oracle's.  Attention's
tolerance, u = 2^-11 (weights x V scale are rounded to f16, the sum of weights
is not):
* every product of a weight is off by u relative: u sum w |V|;
* weights are multiples of 2^-16 units, rounded: off by 2^-17, and a row's largest is
  at least 2^10 units: L keys of at most 448 are off by L 448 2^-27 of the largest V scale;
* scores: a float32 sum of D products is off by at most D 2^-23 sum |q K|
  scale; q's values go down to 2^-31 of the row's largest.  A score moves its
  weight and the sum of weights by that much relative;
* 16-bit outputs: half a step.
"""
import numpy as np
import pytest
import torch

from oracle import scaled as O
from paged_kv_cache_191_gb300 import ops, workloads as W
from tests.gpu_util import half_ulp, held_by_a_call_on_another_stream, requires_cuda
from tests.scaled_inputs import Drafts, ScaledBatch

pytestmark = [pytest.mark.gpu, requires_cuda]
DEV = "cuda"
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def no_device_errors():
    ops.device_errors(clear=True)
    yield
    assert ops.device_errors(clear=True) == 0, "kernel flagged a device error"


def dev(x):
    return (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).to(DEV)


def caches(w):
    return [dev(w.k).view(F8), dev(w.v).view(F8), dev(w.k_scale), dev(w.v_scale)]


def as_np(cs):
    return [c.view(torch.uint8).cpu().numpy() if c.dtype == F8 else c.cpu().numpy() for c in cs]


# ---- append ------------------------------------------------------------------
def append(w, cs, packed=False, stream=None):
    k, v = dev(w.new_k), dev(w.new_v)
    if packed:  # views of one projection
        k, v = torch.cat([k, k, v], 1)[:, w.Hkv:].split([w.Hkv, w.Hkv], 1)
    ops.block_scaled_append(k, v, dev(w.q_start), dev(w.tables), dev(w.lens), *cs, stream=stream)
    return cs


def append_oracle(w):
    return O.append(w.k, w.v, w.k_scale, w.v_scale, w.new_k.double().numpy(), w.new_v.double().numpy(), w.q_start,
                    w.tables, w.lens)


def same(got, want):
    for g, x, name in zip(as_np(got), want, ("k codes", "v codes", "k scale", "v scale")):
        assert np.array_equal(g, x, equal_nan=True), name


BATCHES = [  # new tokens, lengths
    ([1], [1]), ([1], [33]), ([5, 0, 33, 1], [5, 40, 300, 129]), ([17, 64, 15, 16, 18], [17, 70, 30, 48, 33]),
    ([1] * 70, list(range(1, 71))), ([0, 2, 0], [3, 2, 0])]


@pytest.mark.parametrize("Hkv", [1, 5, 8])
@pytest.mark.parametrize("bi", range(len(BATCHES)))
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
def test_append(bi, Hkv, dtype):
    w = ScaledBatch(bi, Hkv, Hkv, *BATCHES[bi], dtype=dtype)
    want = append_oracle(w)
    same(append(w, caches(w)), want)
    same(append(w, caches(w), packed=True), want)


def test_append_grows_and_starts_afresh():
    """Scales far below and far above the new values' own."""
    for s in (2.0 ** -30, 2.0 ** 12):
        w = ScaledBatch(7, 4, 4, [3, 20, 1, 1], [21, 40, 16, 17])
        w.k_scale[:] = w.v_scale[:] = s
        same(append(w, caches(w)), append_oracle(w))


def test_append_of_unusual_values():
    w = ScaledBatch(8, 3, 3, [16, 4, 2], [16, 30, 9], dtype=torch.float32)
    w.new_k[0, 0, 3], w.new_k[1, 0, 5], w.new_k[2, 0, 7] = float("inf"), float("-inf"), float("nan")
    w.new_k[:16, 1] = 0.0
    w.new_k[:16, 2] = 1e-42
    w.new_v[:16, 0] = 3.4e38
    w.new_v[16:20, 1] = float("nan")
    w.new_v[16:20, 2] = float("inf")
    w.new_v[20:, :] = 0.0
    got, want = as_np(append(w, caches(w))), append_oracle(w)
    for i in (0, 1):  # NaN has two codes
        a, b = got[i].copy(), want[i].copy()
        a[(a & 0x7F) == 0x7F] = b[(b & 0x7F) == 0x7F] = 0x7F
        assert np.array_equal(a, b)
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])


def test_append_leaves_everything_else():
    w = ScaledBatch(9, 2, 2, [2, 3], [20, 35])
    before = [w.k.copy(), w.v.copy(), w.k_scale.copy(), w.v_scale.copy()]
    got = as_np(append(w, caches(w)))
    for i in (0, 1):
        rows = np.ones(w.k.shape[:1] + (16,), bool)
        for b, L in enumerate(w.lens):
            for t in range((L - w.sizes[b]) // 16 * 16, L):
                rows[w.tables[b][t // 16], t % 16] = False
        assert np.array_equal(got[i].transpose(0, 2, 1, 3)[rows], before[i].transpose(0, 2, 1, 3)[rows])


@pytest.mark.parametrize("kept", [9, 16])
def test_what_refused_rows_leave(kept):
    """Rows stay, two with large values are appended, refused and written over.  Behind a full block nothing of them is
    left; inside one the block keeps the scale that they raised, and the rows before them are rounded by it."""
    w = ScaledBatch(112, 2, 2, [kept + 2], [kept + 2])
    w.new_k[kept:, :, 3] = 3000.0
    k, v, tables = dev(w.new_k), dev(w.new_v), dev(w.tables)
    cs, clean = caches(w), caches(w)
    state = [w.k, w.v, w.k_scale, w.v_scale]

    def step(to, lo, n, kk, vv):
        q, L = dev(np.array([0, n], dtype=np.int32)), dev(np.array([lo + n], dtype=np.int32))
        ops.block_scaled_append(kk, vv, q, tables, L, *to)
        return O.append(*state, kk.cpu().double().numpy(), vv.cpu().double().numpy(), [0, n], w.tables, [lo + n])

    small = k[:1] * 0.5
    for to in (cs, clean):
        state = [w.k, w.v, w.k_scale, w.v_scale]
        state = step(to, 0, kept, k[:kept], v[:kept])
        if to is cs:
            state = step(to, kept, 2, k[kept:], v[kept:])
            same(to, state)
        state = step(to, kept, 1, small, v[:1])
        same(to, state)
    a, b = as_np(cs), as_np(clean)
    first, last = w.tables[0][0], w.tables[0][kept // 16]
    if kept == 16:
        rows = np.s_[:, :1]  # the row that took the refused ones' place
        assert all(np.array_equal(x[first], y[first]) for x, y in zip(a, b))
        assert all(np.array_equal(x[last][rows], y[last][rows]) for x, y in zip(a[:2], b[:2]))
        assert all(np.array_equal(x[last], y[last]) for x, y in zip(a[2:], b[2:]))
    else:
        assert (a[2][first] == 2.0 ** 3).all() and (b[2][first] < 2.0 ** -5).all()
        x, y = (O.gather(c[0], c[2], w.tables[0], kept, 0) for c in (a, b))
        assert (x != y).any() and (np.abs(x - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** 3)).all()


def test_append_flags_what_it_cannot_store():
    w = ScaledBatch(10, 2, 2, [2, 3, 4], [20, 35, 18])
    good = append_oracle(w)
    for what in ("block", "length", "q_start"):
        x = ScaledBatch(10, 2, 2, [2, 3, 4], [20, 35, 18])
        if what == "block":
            x.tables[1][2] = 10 ** 6
        elif what == "length":
            x.lens[1] = 10 ** 6
        else:
            x.q_start = np.array([0, 5, 2, 9], dtype=np.int32)
        got = as_np(append(x, caches(x)))
        want = {"block": ops.DEVERR_BLOCK_RANGE, "length": ops.DEVERR_CONTEXT_LEN, "q_start": ops.DEVERR_QUERY_RANGE}
        assert ops.device_errors(clear=True) & want[what]
        if what != "q_start":
            for b in (0, 2):
                for g, y in zip(got, good):
                    ids = w.tables[b][:-(-w.lens[b] // 16)]
                    assert np.array_equal(g[ids], y[ids])


def test_append_of_a_q_start_out_of_order():
    """Flagged; what is stored of the batch's other sequences is theirs, and no other row or block is written."""
    w = ScaledBatch(11, 2, 2, [100, 3, 50], [120, 35, 70])
    good = append_oracle(w)
    x = ScaledBatch(11, 2, 2, [100, 3, 50], [120, 35, 70])
    before = [x.k.copy(), x.v.copy(), x.k_scale.copy(), x.v_scale.copy()]
    x.q_start = np.array([50, 150, 0, 50], dtype=np.int32)
    for t, o in ((x.new_k, w.new_k), (x.new_v, w.new_v)):
        t[50:150], t[:50] = o[:100], o[103:]
    got = as_np(append(x, caches(x)))
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE
    for b in range(len(w.k)):
        for g, old, new in zip(got, before, good):
            mine = any(b in w.tables[s][:-(-w.lens[s] // 16)] for s in (0, 2))
            assert np.array_equal(g[b], old[b]) or (mine and np.array_equal(g[b], new[b]))


# ---- attention -----------------------------------------------------------------
def attend(w, cs=None, out_dtype=torch.float32, q=None, max_len=None, max_q=None, **kw):
    cs = cs or caches(w)
    q = dev(w.q) if q is None else q
    max_q = max_q or max(1, int(w.sizes.max(initial=0)))
    need = ops.block_scaled_attention_workspace_size(w.Hq, max_q, cs[0])
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN floats: stale scratch must not leak
    out = torch.full(w.q.shape, float("nan"), dtype=out_dtype, device=DEV)
    ops.block_scaled_attention(q, dev(w.q_start), *cs, dev(w.tables), dev(w.lens),
                               max_len or max(1, int(w.lens.max(initial=0))), max_q, w.scale, out=out, workspace=ws,
                               **kw)
    torch.cuda.synchronize()
    return out.cpu()


def attention_oracle(w):
    return O.attention(w.q.double().numpy(), w.q_start, w.k, w.v, w.k_scale, w.v_scale, w.tables, w.lens, w.scale)


def check(out, w, ref=None, what="", rows=None):
    want, spread, score, wide = ref or attention_oracle(w)
    keys = np.repeat(w.lens.astype(np.float64), w.sizes)[:, None, None]
    vs = float(np.nanmax(np.abs(w.v_scale)))
    moved = 2 * (2 * O.D * 2.0 ** -23 * score + 2.0 ** -30 * wide)[..., None] + 2.0 ** -18
    tol = spread * (2.0 ** -11 + moved) + keys * 448 * vs * 2.0 ** -27
    if out.dtype != torch.float32:
        tol = tol + half_ulp(np.abs(want) + tol, out.dtype)
    got = out.double().numpy()
    if rows is not None:
        got, want, tol = got[rows], want[rows], tol[rows]
    assert np.isfinite(got).all(), what
    worst = (np.abs(got - want) / (tol + 1e-30)).max(initial=0.0)
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


SHAPES = [(4, 4), (8, 1), (6, 2), (16, 1), (24, 2), (32, 1), (10, 2), (64, 8)]
ATTEND = [  # new tokens, lengths
    ([1], [1]), ([1] * 9, [1, 16, 17, 127, 128, 129, 255, 256, 300]), ([5, 0, 33, 1], [5, 40, 300, 129]),
    ([2, 3, 4], [128, 130, 640]), ([150, 3], [700, 3])]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bi", range(len(ATTEND)))
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_attention(shape, bi, dtype):
    w = ScaledBatch(20 + bi, *shape, *ATTEND[bi], dtype=dtype)
    ref = attention_oracle(w)
    check(attend(w), w, ref, what=f"{shape} {ATTEND[bi]}")
    check(attend(w, out_dtype=dtype), w, ref, what=f"{shape} {ATTEND[bi]} 16-bit")


@pytest.mark.parametrize("sizes", [[1, 1, 1], [2, 1, 4], [9, 40, 2]])
def test_attention_over_many_ctas(sizes):
    """Long contexts of few sequences: every item is cut over many CTAs."""
    w = ScaledBatch(30, 8, 1, sizes, [6000, 3001, 130])
    check(attend(w), w)


@pytest.mark.parametrize("n,Hq", [(1, 16), (2, 64), (3, 96)])
def test_many_short_pieces_in_a_cta(n, Hq):
    """Items of one and two chunks, a dozen of them and more in every CTA: the
    same bits ten times over, and every row right."""
    lens = [int(x) for x in W.rng_for(31).integers(n, 257, 160)]
    w = ScaledBatch(31, Hq, 16, [n] * 160, lens)
    first = attend(w)
    check(first, w)
    for _ in range(9):
        assert torch.equal(attend(w), first)


def test_attention_reads_a_packed_projection():
    w = ScaledBatch(32, 8, 2, [3, 1], [40, 200])
    q = torch.cat([dev(w.q), dev(w.q)[:, :4]], 1)[:, :8]
    assert not q.is_contiguous()
    assert torch.equal(attend(w, q=q), attend(w))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_of_the_scores(scale):
    w = ScaledBatch(33, 8, 2, [3, 1], [40, 300])
    w.scale = scale
    check(attend(w), w)


def test_large_and_small_queries():
    """A row of large values beside rows of small ones, in bf16's range: each
    keeps its own precision."""
    w = ScaledBatch(34, 8, 1, [2, 2], [100, 260], dtype=torch.bfloat16)
    w.q[0, 0] *= 2.0 ** 60
    w.q[0, 1] *= 2.0 ** -30
    w.q[1, 3] *= 2.0 ** -100
    w.q[2, 2] = 0.0
    w.k_scale[:] = 2.0 ** -7
    ref = attention_oracle(w)
    rows = np.ones(w.q.shape[:2], bool)
    rows[0, 0] = False  # (its scores differ by more than a float32 product is exact to)
    check(attend(w), w, ref, rows=rows)


@pytest.mark.parametrize("n", [1, 4, 5, 20])
def test_large_queries_over_small_keys(n):
    """bf16 queries near 2^124 and K scales near 2^-124: their products are of the usual size, though a query's sum
    with the codes alone is beyond float32."""
    w = ScaledBatch(113, 8, 1, [n, n], [100, 260], dtype=torch.bfloat16)
    w.q *= 2.0 ** 124
    w.k_scale *= 2.0 ** -117
    w.scale *= 0.5
    check(attend(w), w)


@pytest.mark.parametrize("vs", [2.0 ** -60, 2.0 ** -14, 2.0 ** 10])
def test_v_scales_of_any_size(vs):
    w = ScaledBatch(35, 8, 2, [1, 5], [400, 700])
    w.v_scale[:] = vs * np.where(W.rng_for(3).random(w.v_scale.shape) < 0.3, 0.25, 1.0)
    check(attend(w), w)


def test_a_tail_of_many_small_weights():
    """One key far above thousands of equal ones, whose sum still counts."""
    w = ScaledBatch(36, 4, 1, [1], [20000])
    w.k[:], w.k_scale[:] = 0, 1.0
    w.q[:] = 1.0
    blk = w.tables[0][3]
    w.k[blk, 0, 5] = 0x38  # 1.0 in every dim: 128 above the others
    for top in (4.0, 8.0, 11.0):
        w.scale = top / 128
        check(attend(w), w, what=f"{top}")


def test_maxima_that_keep_growing():
    """Scores that rise along the context, so that every chunk moves the references."""
    w = ScaledBatch(37, 8, 1, [1, 2], [3000, 1500])
    w.q[:] = 1.0
    for b, L in enumerate(w.lens):
        for j, blk in enumerate(w.tables[b][:-(-L // 16)]):
            w.k[blk], w.k_scale[blk] = 0x38, 2.0 ** -2 * (1 + j)
    w.scale = 0.02
    check(attend(w), w)


@pytest.mark.parametrize("n", [1, 3, 20])
def test_stale_rows_are_not_read(n):
    """NaN codes and scales wherever no token may look: behind the contexts, in
    free blocks, and in the later tokens of a chain."""
    w = ScaledBatch(38, 8, 2, [n, n, n], [n, 37, 260], spare=5)
    used = np.zeros(w.k.shape[:1], bool)
    ref = attention_oracle(w)
    for b, L in enumerate(w.lens):
        ids = w.tables[b][:-(-L // 16)]
        used[ids] = True
        if L % 16:
            w.k[ids[-1], :, L % 16:] = w.v[ids[-1], :, L % 16:] = 0x7F
    w.k[~used] = w.v[~used] = 0xFF
    w.k_scale[~used] = w.v_scale[~used] = np.nan
    out = attend(w)
    check(out, w, ref)
    if n > 1:  # a NaN row of the last token reaches no other
        last = w.q_start[1:] - 1
        for b, L in enumerate(w.lens):
            blk = w.tables[b][(L - 1) // 16]
            w.k[blk, :, (L - 1) % 16] = 0x7F
            w.v[blk, :, (L - 1) % 16] = 0x7F
        got = attend(w)
        rows = np.ones(w.q.shape[:2], bool)
        rows[last] = False
        check(got, w, ref, rows=rows)
        assert torch.isnan(got[torch.from_numpy(last).long()]).all()


def test_a_nan_value_reaches_its_dim_only():
    w = ScaledBatch(39, 8, 2, [4], [50])
    ref = attention_oracle(w)
    blk = w.tables[0][2]
    w.v[blk, 1, 47 - 32, 9] = 0x7F  # token 1 of the chain (position 47), kv head 1, dim 9
    got = attend(w)
    nan = torch.isnan(got).numpy()
    want = np.zeros_like(nan)
    want[1:, 4:, 9] = True
    assert np.array_equal(nan, want)
    got[torch.from_numpy(nan)] = torch.from_numpy(ref[0])[torch.from_numpy(nan)].float()
    check(got, w, ref)


def test_a_nan_query_stays_in_its_row():
    w = ScaledBatch(40, 8, 2, [2], [90])
    ref = attention_oracle(w)
    w.q[0, 2, 7], w.q[1, 5, 0] = float("nan"), float("inf")
    got = attend(w)
    rows = np.ones(w.q.shape[:2], bool)
    rows[0, 2] = rows[1, 5] = False
    check(got, w, ref, rows=rows)
    assert torch.isnan(got[0, 2]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_many_short_items_of_a_row_a_thread(dtype):
    """96 rows a kv head, one and two chunks, more than a dozen items in every CTA."""
    lens = [int(x) for x in W.rng_for(47).integers(12, 257, 100)]
    w = ScaledBatch(47, 128, 16, [12] * 100, lens, dtype=dtype)
    first = attend(w)
    check(first, w)
    for _ in range(9):
        assert torch.equal(attend(w), first)


def test_bf16_queries_of_any_size_in_a_prompt():
    """Rows of large, small and no values, and of no numbers, beside each other."""
    w = ScaledBatch(48, 8, 1, [20, 45], [100, 260], dtype=torch.bfloat16)
    w.k_scale[:] = 2.0 ** -7
    w.q[3, 1] *= 2.0 ** -30
    w.q[5, 3] *= 2.0 ** -100
    w.q[5, 4] *= 2.0 ** -126
    w.q[30, 2] = 0.0
    w.q[40, 0, :3] *= 2.0 ** 3
    ref = attention_oracle(w)
    check(attend(w), w, ref)
    rows = np.ones(w.q.shape[:2], bool)
    w.q[0, 0] *= 2.0 ** 60  # (its scores differ by more than a float32 product is exact to)
    w.q[7, 2, 9], w.q[33, 5, 0] = float("nan"), float("inf")
    rows[0, 0] = rows[7, 2] = rows[33, 5] = False
    got = attend(w)
    kept = torch.from_numpy(rows)
    assert torch.isnan(got[7, 2]).all() and torch.isnan(got[33, 5]).all()
    w.q[0, 0], w.q[7, 2], w.q[33, 5] = 1.0, 1.0, 1.0
    again = attend(w)
    check(again, w)
    assert torch.equal(again[kept], got[kept])


def test_attention_flags_and_clamps():
    w = ScaledBatch(41, 8, 2, [2, 1, 3], [40, 20, 33])
    ref = attention_oracle(w)
    w.tables[1][1] = -5  # block 0 is read instead
    out = attend(w)
    assert ops.device_errors(clear=True) == ops.DEVERR_BLOCK_RANGE
    rows = np.ones(w.q.shape[:2], bool)
    rows[2] = False
    check(out, w, ref, rows=rows)
    w.tables[1][1] = 0
    out = attend(w, max_q=2)  # the third sequence is too long: skipped
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE
    check(out, w, ref, rows=rows & (np.arange(6) < 3)[:, None])
    assert torch.isnan(out[3:]).all()
    x = ScaledBatch(42, 8, 2, [5], [3])  # more tokens than the context has: the first two see nothing
    out = attend(x)
    assert ops.device_errors(clear=True) == ops.DEVERR_CONTEXT_LEN
    check(out, x)
    assert (out[:2] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("n,L", [(300, 100), (1024, 100), (700, 300)])
def test_a_prompt_of_more_tokens_than_keys(n, L, dtype):
    """Above 40 rows a kv head: the tokens without a key are zero rows, and no other row stays unwritten."""
    w = ScaledBatch(100, 32, 8, [n, 3], [L, 60], dtype=dtype)
    ref = attention_oracle(w)
    for out_dtype in (torch.float32, dtype):
        out = attend(w, out_dtype=out_dtype)
        assert ops.device_errors(clear=True) == ops.DEVERR_CONTEXT_LEN
        check(out, w, ref)
        assert (out[:n - L] == 0).all()


# ---- the thread-per-row kernel (above 40 rows of a kv head) where the values are unusual ----
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_of_a_prompts_scores(scale, dtype):
    w = ScaledBatch(101, 8, 2, [30, 11], [40, 300], dtype=dtype)
    w.scale = scale
    check(attend(w), w)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("vs", [2.0 ** -60, 2.0 ** -14, 2.0 ** 10])
def test_v_scales_of_any_size_in_a_prompt(vs, dtype):
    w = ScaledBatch(102, 8, 2, [25, 45], [400, 700], dtype=dtype)
    w.v_scale[:] = vs * np.where(W.rng_for(3).random(w.v_scale.shape) < 0.3, 0.25, 1.0)
    check(attend(w), w)


def test_a_tail_of_many_small_weights_in_a_prompt():
    w = ScaledBatch(103, 4, 1, [20], [20000])
    w.k[:], w.k_scale[:] = 0, 1.0
    w.q[:] = 1.0
    w.k[w.tables[0][3], 0, 5] = 0x38
    for top in (4.0, 8.0, 11.0):
        w.scale = top / 128
        check(attend(w), w, what=f"{top}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_maxima_that_keep_growing_in_a_prompt(dtype):
    w = ScaledBatch(104, 8, 1, [20, 90], [3000, 1500], dtype=dtype)
    w.q[:] = 1.0
    for b, L in enumerate(w.lens):
        for j, blk in enumerate(w.tables[b][:-(-L // 16)]):
            w.k[blk], w.k_scale[blk] = 0x38, 2.0 ** -2 * (1 + j)
    w.scale = 0.02
    check(attend(w), w)


def test_a_nan_query_stays_in_its_row_of_a_prompt():
    w = ScaledBatch(105, 8, 2, [40], [90])
    ref = attention_oracle(w)
    w.q[0, 2, 7], w.q[31, 5, 0] = float("nan"), float("nan")
    got = attend(w)
    rows = np.ones(w.q.shape[:2], bool)
    rows[0, 2] = rows[31, 5] = False
    check(got, w, ref, rows=rows)
    assert torch.isnan(got[0, 2]).all() and torch.isnan(got[31, 5]).all()


def test_a_nan_value_reaches_its_dim_only_in_a_prompt():
    w = ScaledBatch(106, 8, 2, [40], [50])
    ref = attention_oracle(w)
    blk = w.tables[0][2]
    w.v[blk, 1, 47 - 32, 9] = 0x7F  # position 47, token 37
    got = attend(w)
    nan = torch.isnan(got).numpy()
    want = np.zeros_like(nan)
    want[37:, 4:, 9] = True
    assert np.array_equal(nan, want)
    got[torch.from_numpy(nan)] = torch.from_numpy(ref[0])[torch.from_numpy(nan)].float()
    check(got, w, ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_a_prompt_reads_a_packed_projection_and_leaves_the_rows_behind(dtype):
    w = ScaledBatch(107, 8, 2, [33, 1], [40, 200], dtype=dtype)
    want = attend(w)
    q = torch.cat([dev(w.q), dev(w.q)[:, :4]], 1)[:, :8]
    assert not q.is_contiguous() and torch.equal(attend(w, q=q), want)
    w.q = torch.cat([w.q, w.q])
    got = attend(w)
    assert torch.equal(got[:34], want) and torch.isnan(got[34:]).all()


def test_decode_steps_in_a_call_for_prompts():
    """Single tokens beside one prompt, and alone in a call that allows prompts."""
    w = ScaledBatch(109, 32, 8, [1] * 12 + [90, 0, 1], [1, 15, 16, 17, 128, 129, 300, 511, 700, 1030, 64, 2, 400, 33, 256])
    check(attend(w), w)
    x = ScaledBatch(110, 32, 8, [1] * 6, [1, 16, 129, 300, 700, 1030])
    check(attend(x, max_q=500), x)


# ---- both kernels, and the calls in graphs and on streams ----
def test_rows_behind_the_last_sequence_stay():
    w = ScaledBatch(43, 8, 2, [2, 1], [40, 20])
    want = attend(w)
    w.q = torch.cat([w.q, w.q])
    got = attend(w)
    assert torch.equal(got[:3], want) and torch.isnan(got[3:]).all()


def test_calls_replay_in_a_graph():
    """Append, attention and verification captured once and replayed on new
    values of the same buffers."""
    w = ScaledBatch(44, 8, 2, [3, 2], [40, 300])
    d = Drafts(44, [3, 2], 1000, "sampled")
    cs, k, v, q = caches(w), dev(w.new_k), dev(w.new_v), dev(w.q)
    qs, tables, lens = dev(w.q_start), dev(w.tables), dev(w.lens)
    tok, p, u, dr = (dev(x) for x in (d.tokens, d.target, d.uniform, d.draft))

    def step():
        ops.block_scaled_append(k, v, qs, tables, lens, *cs)
        out = ops.block_scaled_attention(q, qs, *cs, tables, lens, 300, 3, w.scale)
        return out, *ops.draft_verify(tok, p, u, qs, 3, draft_probs=dr)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (1, 2):
        x, e = ScaledBatch(50 + seed, 8, 2, [3, 2], [40, 300]), Drafts(50 + seed, [3, 2], 1000, "sampled")
        for a, b in ((k, x.new_k), (v, x.new_v), (q, x.q), (tok, e.tokens), (p, e.target), (u, e.uniform), (dr, e.draft)):
            a.copy_(dev(b))
        g.replay()
        first = [t.clone() for t in got]
        for a, b in zip(step(), first):
            assert torch.equal(a, b)


def test_calls_on_another_stream(monkeypatch):
    w = ScaledBatch(45, 8, 2, [3, 2], [40, 300])
    cs, args = caches(w), (dev(w.q_start), dev(w.tables), dev(w.lens))
    q = dev(w.q)
    call = lambda st: [ops.block_scaled_attention(q, args[0], *cs, args[1], args[2], 300, 3, w.scale, stream=st)]  # noqa: E731
    plain, other = held_by_a_call_on_another_stream(monkeypatch, ops, call)
    assert torch.equal(plain[0], other[0])


def test_verification_on_another_stream(monkeypatch):
    d = Drafts(46, [3, 1, 5], 5000, "sampled")
    a = [dev(x) for x in (d.tokens, d.target, d.uniform, d.q_start)]
    dr = dev(d.draft)
    plain, other = held_by_a_call_on_another_stream(
        monkeypatch, ops, lambda st: list(ops.draft_verify(*a, 5, draft_probs=dr, stream=st)))
    for x, y in zip(plain, other):
        assert torch.equal(x, y)


# (query heads, tokens) over one kv head: 8, 16, 32 and 40 rows of an item, a thread per row
KERNELS = [(8, 1), (16, 1), (8, 4), (8, 5), (32, 9)]


def test_kernels_take_turns_in_one_workspace():
    """One long item each, cut over most CTAs, in a workspace that holds what the
    call before left there."""
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    first = {}
    for turn in range(3):
        for i, (Hq, n) in enumerate(KERNELS):
            w = ScaledBatch(70 + i, Hq, 1, [n], [9000 + 1111 * i])
            cs = caches(w)
            out = ops.block_scaled_attention(dev(w.q), dev(w.q_start), *cs, dev(w.tables), dev(w.lens),
                                             int(w.lens[0]), n, w.scale, out_dtype=torch.float32, workspace=ws).cpu()
            if turn == 0:
                check(out, w, what=f"{Hq} heads, {n} tokens")
            assert torch.equal(first.setdefault(i, out), out)


def test_graphs_share_a_workspace():
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    runs = []
    for i, (Hq, n) in enumerate(KERNELS):
        w = ScaledBatch(80 + i, Hq, 1, [n, n], [5000, 700])
        a = [dev(w.q), dev(w.q_start), *caches(w), dev(w.tables), dev(w.lens)]
        want = ops.block_scaled_attention(*a, 5000, n, w.scale, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = ops.block_scaled_attention(*a, 5000, n, w.scale, workspace=ws)
        runs.append((g, got, want, a))  # (a graph reads its operands where they were)
    for order in (range(5), (4, 0, 3, 3, 1, 0, 2), range(4, -1, -1)):
        for i in order:
            runs[i][1].fill_(float("nan"))
            runs[i][0].replay()
        for i in order:
            assert torch.equal(runs[i][1], runs[i][2])


def test_blocks_beyond_32_bits():
    """Blocks at the end of pools of 2^31 bytes and more hold and give what they do at the start."""
    w = ScaledBatch(48, 16, 16, [3, 18], [100, 50])
    cs, n = caches(w), len(w.k)
    far = 2 ** 31 // (16 * 2048) + 4000
    big = [torch.zeros((far + n, *c.shape[1:]), dtype=torch.uint8 if c.dtype == F8 else c.dtype, device=DEV) for c in cs]
    big = [b.view(F8) if c.dtype == F8 else b for b, c in zip(big, cs)]
    ops.block_scaled_copy(*big, *cs, dev(np.array([[i, far + i] for i in range(n)], dtype=np.int64)))
    append(w, cs)
    want = attend(w, cs)
    w.tables = np.where(w.tables >= 0, w.tables + far, w.tables).astype(np.int32)
    append(w, big)
    assert torch.equal(attend(w, big), want)
    same([b[far:] for b in big], as_np(cs))


@pytest.mark.parametrize("Hq,n", [(8, 1), (8, 5), (32, 9)])
def test_no_tokens(Hq, n):
    """Sequences without new tokens, and tensors without elements."""
    w = ScaledBatch(49, Hq, 2, [0, 0], [40, 3])
    for t in (w.q, w.new_k, w.new_v):
        assert t.numel() == 0
    cs = caches(w)
    same(append(w, cs), [w.k, w.v, w.k_scale, w.v_scale])
    assert attend(w, cs, max_q=n).shape == (0, Hq, 128)
    e = ScaledBatch(49, Hq, 2, [n], [40])
    e.q_start, e.tables, e.lens = e.q_start[:1], e.tables[:0], e.lens[:0]
    same(append(e, cs), [w.k, w.v, w.k_scale, w.v_scale])
    assert torch.isnan(attend(e, cs, max_len=40, max_q=n)).all()
    d = Drafts(49, [0, 0], 30, "sampled")
    path, k, tok = verify(d, 3)
    assert (path == -1).all() and (k == 0).all() and (tok == -1).all()


def test_append_and_copy_on_another_stream():
    w = ScaledBatch(45, 8, 2, [3, 2], [40, 300])
    cs, want = caches(w), append_oracle(w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pairs = dev(np.array([[0, len(w.k) - 1]], dtype=np.int64))
    k, v, a = dev(w.new_k), dev(w.new_v), [dev(x) for x in (w.q_start, w.tables, w.lens)]
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    ops.block_scaled_append(k, v, *a, *cs, stream=s)
    assert not s.query()
    ops.block_scaled_copy(*cs, *cs, pairs, stream=s)
    s.synchronize()
    for x in want:
        x[-1] = x[0]
    same(cs, want)


# ---- copies --------------------------------------------------------------------
@pytest.mark.parametrize("Hkv", [1, 5, 40])
def test_copy_within_and_between_pools(Hkv):
    w = ScaledBatch(47, Hkv, Hkv, [1], [160])
    cs = caches(w)
    pairs = np.array([[0, 5], [3, 1], [0, 2]], dtype=np.int64)
    ops.block_scaled_copy(*cs, *cs, dev(pairs))
    want = [w.k.copy(), w.v.copy(), w.k_scale.copy(), w.v_scale.copy()]
    for x in want:
        x[[5, 1, 2]] = x[[0, 3, 0]]
    same(cs, want)
    host = [torch.zeros((4, *c.shape[1:]), dtype=c.dtype).pin_memory() for c in cs]
    ops.block_scaled_copy(*host, *cs, dev(np.array([[7, 0], [2, 3]], dtype=np.int64)))
    torch.cuda.synchronize()
    for h, x in zip(as_np(host), want):
        assert np.array_equal(h[[0, 3]], x[[7, 2]]) and not h[1:3].any()
    ops.block_scaled_copy(*cs, *host, dev(np.array([[0, 99], [4, 0], [3, 6]], dtype=np.int64)))
    assert ops.device_errors(clear=True) == ops.DEVERR_BLOCK_RANGE
    for x in want:
        x[6] = x[2]
    same(cs, want)


def test_two_calls_at_once():
    """Calls on two streams, each with the workspace that it allocates."""
    runs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i, (Hq, n) in enumerate([(8, 1), (8, 5), (32, 9)]):
        w = ScaledBatch(90 + i, Hq, 1, [n, n, n], [5000, 700, 129])
        a = [dev(w.q), dev(w.q_start), *caches(w), dev(w.tables), dev(w.lens), 5000, n, w.scale]
        runs.append((a, ops.block_scaled_attention(*a)))
    torch.cuda.synchronize()
    got = []
    for turn in range(12):
        a, want = runs[turn % 3]
        got += [(ops.block_scaled_attention(*a, stream=st), want) for st in streams]
    torch.cuda.synchronize()
    for x, want in got:
        assert torch.equal(x, want)


# ---- verification --------------------------------------------------------------
def verify(d, max_path, strided=False):
    t, q = dev(d.target), None if d.draft is None else dev(d.draft)
    if strided:  # rows of a wider buffer, at odd places
        T, V = t.shape
        t = torch.cat([torch.full((T, 3), 9.0, device=DEV), t, torch.full((T, 2), 9.0, device=DEV)], 1)[:, 3:3 + V]
        q = None if q is None else torch.cat([torch.full((T, 1), 9.0, device=DEV), q], 1)[:, 1:]
    path, n, tok = ops.draft_verify(dev(d.tokens), t, dev(d.uniform), dev(d.q_start), max_path, draft_probs=q,
                                    parents=None if d.parents is None else dev(d.parents))
    return path.cpu().numpy(), n.cpu().numpy(), tok.cpu().numpy()


def check_verify(got, d, max_path):
    paths, nexts = O.verify(d.tokens, d.target, d.uniform, d.q_start, max_path, d.draft, d.parents)
    path, n, tok = got
    assert n.tolist() == [len(p) for p in paths]
    for b, p in enumerate(paths):
        assert path[b].tolist() == p + [-1] * (max_path - len(p))
    assert tok.tolist() == nexts


@pytest.mark.parametrize("kind", ["sampled", "picked", "tree"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099, 50001])
def test_verify(kind, V):
    sizes = [1, 5, 0, 9, 3, 2, 7, 40] * (4 if V < 5000 else 1)
    d = Drafts(V, sizes, V, kind)
    check_verify(verify(d, 40), d, 40)
    check_verify(verify(d, 3, strided=True), d, 3)
    check_verify(verify(d, 1), d, 1)


@pytest.mark.parametrize("kind", ["picked", "tree"])
def test_verify_of_many_children(kind):
    """Hundreds of nodes, many below one parent, tokens that repeat."""
    d = Drafts(3, [1024, 300, 70], 40, kind, sharp=0.3)
    if kind == "tree":
        d.parents[1:600] = 0
    check_verify(verify(d, 50), d, 50)


def test_verify_of_many_sequences():
    """More sequences than the SMs have warps for."""
    d = Drafts(11, [2, 1, 3, 0, 1] * 1400, 300, "sampled")
    check_verify(verify(d, 3), d, 3)


def test_verify_of_the_largest_vocabulary():
    V = 1 << 19
    d = Drafts(12, [2, 3], V, "sampled")
    d.uniform[0], d.uniform[2] = 1.0 - 2.0 ** -24, 0.5
    check_verify(verify(d, 3), d, 3)
    d.draft = None
    check_verify(verify(d, 3), d, 3)


def test_verify_refuses_what_it_cannot_read():
    d = Drafts(13, [2, 3], 100, "sampled")
    tok, p, u, qs = (dev(x) for x in (d.tokens, d.target, d.uniform, d.q_start))
    bad = [dict(target_probs=p[:1].expand(5, 100)), dict(target_probs=p.double()), dict(target_probs=p.t()),
           dict(target_probs=torch.empty(5, 0, device=DEV)), dict(draft_probs=p[:, :99]), dict(tokens=tok.int()),
           dict(uniform=u[:4]), dict(parents=torch.zeros(5, dtype=torch.int64, device=DEV)),
           dict(parents=torch.zeros(5, dtype=torch.int32, device=DEV), draft_probs=p),
           dict(target_probs=torch.empty(5, (1 << 19) + 1, device=DEV)), dict(max_path=0)]
    for kw in bad:
        with pytest.raises((ValueError, RuntimeError)):
            ops.draft_verify(**(dict(tokens=tok, target_probs=p, uniform=u, q_start=qs, max_path=3) | kw))


def test_verify_edges_of_the_draw():
    """u0 at the ends of its range, ties at a sum, weights too small to count."""
    d = Drafts(4, [1] * 8, 4, "picked")
    d.target[:] = np.array([0.25, 0.5, 0.0, 0.25], dtype=np.float32)
    d.uniform[:] = [0.0, 0.25, np.nextafter(np.float32(0.25), np.float32(0)), 0.75, 1.0 - 2.0 ** -24, 0.5, 1.0, np.nan]
    check_verify(verify(d, 2), d, 2)
    assert verify(d, 2)[2].tolist() == [0, 1, 0, 3, 3, 1, 3, 0]
    d.target[:] = np.array([0.0, 2.0 ** -50, 2.0 ** -44, 0.0], dtype=np.float32)
    assert verify(d, 2)[2].tolist() == [2] * 8


def test_verify_draws_from_the_exact_sum():
    """u0 times the sum lies just below a whole number that is also a cumulated sum, nearer than a float64 product
    tells; and a sum of 2^54 - 1, which float64 has not."""
    d = Drafts(14, [1, 1], 1026, "picked")
    d.target[:] = 0.0
    # 8393261 2^20 = u0 x sum + 1866 2^-24, in units of 2^-44
    m, first, rest = 11191015, 8393261 << 20, 4393167093978
    assert m * (first + rest) == (first << 24) - 1866
    d.target[0, :3] = np.array([first, rest >> 20 << 20, rest & 0xFFFFF], dtype=np.float64) * 2.0 ** -44
    d.target[1, :1023], d.target[1, 1023], d.target[1, 1024] = 1.0, 1.0 - 2.0 ** -24, (2 ** 20 - 1) * 2.0 ** -44
    d.uniform[:] = [m * 2.0 ** -24, 0.5]
    assert sum(int(x * 2.0 ** 44) for x in d.target[0].astype(np.float64)) == first + rest
    assert sum(int(x * 2.0 ** 44) for x in d.target[1].astype(np.float64)) == 2 ** 54 - 1
    got = verify(d, 2)
    assert got[2].tolist() == [0, 511]
    check_verify(got, d, 2)


def test_verify_where_nothing_is_left():
    d = Drafts(5, [2, 2, 1], 50, "sampled")
    d.draft[:] = 1.0  # takes everything: the target's own row
    d.uniform[:] = 0.999
    check_verify(verify(d, 2), d, 2)
    d.target[4] = 0.0
    got = verify(d, 2)
    assert ops.device_errors(clear=True) == ops.DEVERR_TREE
    assert got[2][2] == -1 and got[1].tolist()[2] == 1
    check_verify(got, d, 2)


def test_verify_of_unusual_probabilities():
    d = Drafts(6, [3, 3, 3], 100, "sampled")
    d.target[0, :50], d.target[3, 5], d.target[6] = np.nan, np.inf, -1.0
    d.target[6, 7] = 5.0
    d.draft[1, 3], d.draft[4] = np.nan, 1e-45
    check_verify(verify(d, 3), d, 3)


def test_verify_flags_bad_input():
    d = Drafts(7, [3, 4], 30, "tree")
    d.parents[5] = 5
    got = verify(d, 4)
    assert ops.device_errors(clear=True) == ops.DEVERR_TREE
    d.parents[5] = -1
    check_verify(got, d, 4)
    d.tokens[1], d.tokens[4] = 30, -7
    got = verify(d, 4)
    assert ops.device_errors(clear=True) == ops.DEVERR_TREE
    check_verify(got, d, 4)
    e = Drafts(8, [3, 1025, 2], 5, "picked")
    got = verify(e, 4)
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE
    assert got[1][1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()
    x = Drafts(8, [3, 1, 2], 5, "picked")
    x.q_start = np.array([0, 5, 3, 6], dtype=np.int32)
    verify(x, 4)
    assert ops.device_errors(clear=True) == ops.DEVERR_QUERY_RANGE


def test_verified_tokens_are_distributed_as_the_target():
    """20000 chains of one row: the tokens behind node 0 have the target's
    shares, within 5 standard deviations."""
    rng = W.rng_for(9)
    B, V = 20000, 12
    p, q = (rng.dirichlet(np.ones(V)).astype(np.float32) for _ in range(2))
    d = Drafts(9, [3], V, "picked")
    d.q_start = (3 * np.arange(B + 1)).astype(np.int32)
    d.target, d.uniform = np.tile(p, (3 * B, 1)), rng.random(3 * B, dtype=np.float32)
    for draft in (np.tile(q, (3 * B, 1)), None):
        d.draft = draft
        q64 = q.astype(np.float64) / q.astype(np.float64).sum()
        d.tokens = rng.choice(V, 3 * B, p=q64) if draft is not None else rng.integers(0, V, 3 * B)
        path, n, tok = verify(d, 3)
        first = np.where(n > 1, d.tokens.reshape(B, 3)[:, 1], tok)
        share = np.bincount(first, minlength=V) / B
        assert (np.abs(share - p) <= 5 * np.sqrt(p / B)).all()


# ---- together ------------------------------------------------------------------
def test_a_sampled_speculative_step():
    """Three steps of four sequences: slots from the block manager, append,
    attention, verification, truncation; two of them share a prompt, whose block
    is copied before it is written."""
    rng = W.rng_for(60)
    Hq, Hkv, V, N = 8, 2, 300, 4
    alloc = ops.BlockAllocator(64)
    lens = [37, 5, 130]
    for i, n in enumerate(lens):
        alloc.alloc_seq(i, n)
    w = ScaledBatch(60, Hq, Hkv, lens, lens)
    tables, ctx = alloc.tables([0, 1, 2], 16)
    w.tables, w.lens = np.ascontiguousarray(tables), np.ascontiguousarray(ctx)
    shape = (64, Hkv, 16, 128)
    w.k, w.v = (np.full(shape, 0x7F, dtype=np.uint8) for _ in range(2))
    w.k_scale, w.v_scale = (np.full(shape[:2], np.nan, dtype=np.float32) for _ in range(2))
    cs = append(w, caches(w))
    state = append_oracle(w)
    same(cs, state)
    alloc.fork(0, 3)
    ids = [0, 1, 2, 3]
    for step in range(3):
        sizes = [int(x) for x in rng.integers(1, N + 1, 4)]
        pairs = []
        for i, n in zip(ids, sizes):
            _, cow = alloc.append_tokens(i, n)
            if cow[0] >= 0:
                pairs.append(cow)
        x = ScaledBatch(61 + step, Hq, Hkv, sizes, [16] * 4)
        tables, ctx = alloc.tables(ids, 16)
        x.tables, x.lens = np.ascontiguousarray(tables), np.ascontiguousarray(ctx)
        x.k, x.v, x.k_scale, x.v_scale = state
        if pairs:
            ops.block_scaled_copy(*cs, *cs, dev(np.array(pairs, dtype=np.int64)))
            for c in state:
                c[[p[1] for p in pairs]] = c[[p[0] for p in pairs]]
        append(x, cs)
        state = append_oracle(x)
        same(cs, state)
        x.k, x.v, x.k_scale, x.v_scale = state
        check(attend(x, cs), x)
        d = Drafts(61 + step, sizes, V, "sampled")
        got = verify(d, N)
        check_verify(got, d, N)
        for i, n, keep in zip(ids, sizes, got[1]):
            alloc.truncate_seq(i, alloc.table(i)[1] - n + int(keep))
