"""The drafted-tree step on the host: the oracle's own pins, the entry
points' refusals, masks from parents, rotary frequencies and the block
manager's truncation.  No GPU."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle.attention import paged_prefill
from oracle import tree as O
from paged_kv_cache_191_gb300 import ops, workloads as W
from tests.libfixture import palib  # noqa: F401
from tests.test_abi import FAKE, _desc
from tests.tree_inputs import TreeBatch, parents_of

INV, UNS, OK = ops.PA_ERR_INVALID, ops.PA_ERR_UNSUPPORTED, ops.PA_OK


# ---- oracle pins -----------------------------------------------------------
def test_chain_mask_is_causal_attention():
    w = TreeBatch(3, 4, 2, 64, "f16", [5, 0, 70], [20, 9, 70])
    for b, n in enumerate(w.sizes):
        for i in range(n):
            row = np.zeros(w.words, np.uint64)
            for j in range(i + 1):
                row[j // 64] |= np.uint64(1) << np.uint64(j % 64)
            w.mask[w.q_start[b] + i] = row.view(np.int64)
    got, spread, score = O.tree_attention(w.q.numpy(), w.q_start, w.mask, w.k.numpy(), w.v.numpy(), w.tables, w.lens,
                                          w.scale)
    want = paged_prefill(w.q.numpy(), w.q_start, w.k.numpy(), w.v.numpy(), w.tables, w.lens, w.scale)
    assert np.allclose(got, want, rtol=0, atol=1e-12)
    assert (spread + 1e-12 >= np.abs(got)).all() and (score >= 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = W.rng_for(4)
    x, pos = rng.standard_normal((7, 3, 64)), rng.integers(0, 5000, 7)
    f, factor = ops.rope_frequencies(32)
    got, mag = O.rotate(x, pos, f.numpy(), 1.5, interleaved)
    z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if interleaved else x[..., :16] + 1j * x[..., 16:32]
    z = z * 1.5 * np.exp(1j * pos[:, None, None] * f.numpy())
    want = x.copy()
    if interleaved:
        want[..., 0:32:2], want[..., 1:32:2] = z.real, z.imag
    else:
        want[..., :16], want[..., 16:32] = z.real, z.imag
    assert np.allclose(got, want, rtol=0, atol=1e-10)
    assert (mag + 1e-9 >= np.abs(got)).all() and np.array_equal(got[..., 32:], x[..., 32:])


def test_acceptance_by_hand():
    # 0 -> 1, 2, 3; 2 -> 4, 5; 5 -> 6
    parents, draft = [-1, 0, 0, 0, 2, 2, 5], [9, 7, 8, 8, 1, 2, 3]
    target = [8, 0, 2, 0, 0, 3, 6]
    assert O.tree_accept(draft, target, parents, [0, 7], 7) == ([[0, 2, 5, 6]], [6])
    assert O.tree_accept(draft, target, parents, [0, 7], 2) == ([[0, 2]], [2])
    assert O.tree_accept(draft, [4] * 7, parents, [0, 7, 7], 7) == ([[0], []], [4, -1])


def test_commit_by_hand():
    k = np.arange(3 * 2 * 16 * 1).reshape(3, 2, 16, 1)
    s = np.arange(48).reshape(3, 16)
    (k2, s2), lens = O.tree_commit([k, s], [[2, 0]], [20], [0, 6], [[0, 3, 5]])
    # the tree is positions 14 .. 19: node 3 (17: block 0, row 1) -> 15, node 5 (19: row 3) -> 16
    assert lens == [17]
    assert np.array_equal(k2[2, :, 15], k[0, :, 1]) and np.array_equal(k2[0, :, 0], k[0, :, 3])
    assert s2[2, 15] == s[0, 1] and s2[0, 0] == s[0, 3] and s2[0, 1] == s[0, 1]


# ---- masks and frequencies -------------------------------------------------
@pytest.mark.parametrize("sizes", [[1], [7, 0, 3], [64, 65], [200]])
def test_tree_mask_lists_ancestors(palib, sizes):
    rng = W.rng_for(sum(sizes))
    par = [parents_of(rng, n) for n in sizes]
    qs = np.concatenate([[0], np.cumsum(sizes)])
    mask, depths = ops.tree_mask(np.concatenate(par), qs)
    assert mask.shape == (sum(sizes), -(-max(sizes) // 64)) and mask.dtype == np.int64
    for b, n in enumerate(sizes):
        for i in range(n):
            up, at = set(), i
            while at >= 0:
                up.add(at)
                at = par[b][at]
            bits = O.visible(mask[qs[b] + i], mask.shape[1] * 64)
            assert set(np.nonzero(bits)[0]) == up and depths[qs[b] + i] == len(up) - 1


def test_tree_mask_refuses(palib):
    for bad in ([-1, 1], [-1, 2, 0], [-2], [0]):
        with pytest.raises(ops.PagedKVError):
            ops.tree_mask(bad)
    with pytest.raises(ValueError):
        ops.tree_mask([-1, 0], [0, 1])
    one = (C.c_int32 * 1)(-1)
    assert palib.pa_tree_mask(one, 1, 0, FAKE, None) == INV
    assert palib.pa_tree_mask(None, 1, 1, FAKE, None) == INV
    assert palib.pa_tree_mask(None, 0, 0, None, None) == OK


def test_rope_frequencies():
    f, a = ops.rope_frequencies(64, base=500000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and a == 1.0 and f[0] == 1.0
    assert math.isclose(float(f[31]), 500000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = ops.rope_frequencies(64, base=500000.0, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    ntk, _ = ops.rope_frequencies(64, scaling="ntk", factor=8.0)
    plain, _ = ops.rope_frequencies(64)
    assert math.isclose(float(ntk[31] * 8), float(plain[31]), rel_tol=1e-12) and ntk[0] == 1.0
    yarn, a = ops.rope_frequencies(64, scaling="yarn", factor=16.0, original_context=4096)
    assert yarn[0] == plain[0] and math.isclose(float(yarn[31]), float(plain[31]) / 16, rel_tol=1e-14)
    assert math.isclose(a, 0.1 * math.log(16.0) + 1.0) and (yarn <= plain).all() and (yarn >= plain / 16).all()
    for kw in ({"scaling": "other"}, {"base": 0.5}, {"factor": 0.5}):
        with pytest.raises(ValueError):
            ops.rope_frequencies(64, **kw)
    for rot in (0, 8, 24):
        with pytest.raises(ValueError):
            ops.rope_frequencies(rot)


# ---- refusals: nothing is launched, so no GPU is needed ------------------------
def _rope(desc, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=ops.F16, qs=512, ks=256, vs=256, pos=FAKE, inv=FAKE, rot=128, inter=0,
             factor=1.0, slots=FAKE, T=3, Hq=4, qo=FAKE + 4096, qdt=ops.F16, os=512, kc=FAKE, vc=FAKE, ksc=None,
             vsc=None)
    a.update(kw)
    return ops.lib().pa_rope_cache_write(
        a["q"], a["k"], a["v"], a["dt"], a["qs"], a["ks"], a["vs"], a["pos"], a["inv"], a["rot"], a["inter"],
        a["factor"], a["slots"], a["T"], a["Hq"], a["qo"], a["qdt"], a["os"], a["kc"], a["vc"], a["ksc"], a["vsc"],
        C.byref(desc), None)


@pytest.mark.parametrize("desc_kw,kw,status", [
    ({}, {"T": 0}, OK), ({"head_dim": 96}, {}, UNS), ({"block_size": 32}, {}, UNS),
    ({}, {"T": -1}, INV), ({}, {"Hq": -1}, INV), ({}, {"rot": 0}, INV), ({}, {"rot": 8}, INV), ({}, {"rot": 144}, INV),
    ({}, {"rot": 40}, INV), ({}, {"inter": 2}, INV), ({}, {"factor": float("inf")}, INV),
    ({}, {"dt": ops.BF16, "qdt": ops.BF16}, INV), ({}, {"dt": ops.FP8_E4M3}, INV), ({}, {"qdt": ops.F32}, INV),
    ({}, {"ksc": FAKE}, INV), ({"kv_dtype": ops.FP8_E4M3}, {}, INV),
    ({"kv_dtype": ops.INT8}, {"ksc": FAKE, "vsc": FAKE + 4}, INV),
    ({}, {"ks": 255}, INV), ({}, {"vs": 260}, INV), ({}, {"qs": 504}, INV), ({}, {"os": 516}, INV),
    ({}, {"q": None}, INV), ({}, {"qo": None}, INV), ({}, {"k": None}, INV), ({}, {"slots": None}, INV),
    ({}, {"inv": None}, INV), ({}, {"pos": FAKE + 4}, INV), ({}, {"k": FAKE + 8}, INV), ({}, {"qo": FAKE + 2}, INV),
    ({}, {"qo": FAKE, "os": 1024}, INV),  # in place with another stride
])
def test_rope_refuses(palib, desc_kw, kw, status):
    assert _rope(_desc(**desc_kw), **kw) == status


def _tree(desc, **kw):
    a = dict(q=FAKE, qdt=ops.F16, qs=FAKE, T=6, mq=4, mask=FAKE, words=1, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE,
             maxb=8, cl=FAKE, maxl=128, B=2, Hq=4, scale=0.1, out=FAKE, odt=ops.F16, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return ops.lib().pa_tree_attention(
        a["q"], a["qdt"], a["qs"], a["T"], a["mq"], a["mask"], a["words"], a["k"], a["v"], a["ks"], a["vs"], a["bt"],
        a["maxb"], a["cl"], a["maxl"], a["B"], a["Hq"], a["scale"], a["out"], a["odt"], C.byref(desc), a["ws"],
        a["wsb"], None)


@pytest.mark.parametrize("desc_kw,kw,status", [
    ({}, {"B": 0}, OK), ({}, {"T": 0, "mq": 0, "words": 0}, OK),
    ({"head_dim": 256}, {}, UNS), ({"kv_dtype": ops.F32}, {}, INV), ({"kv_dtype": ops.INT8, "head_dim": 64}, {}, UNS),
    ({}, {"T": -1}, INV), ({}, {"mq": 0}, INV), ({}, {"mq": 70000, "words": 2000}, UNS), ({}, {"Hq": 3}, INV),
    ({}, {"Hq": 0}, INV), ({}, {"B": -1}, INV), ({}, {"maxl": -1}, INV), ({}, {"maxb": 0}, INV),
    ({}, {"mq": 65}, INV),                       # two mask words needed
    ({}, {"scale": float("nan")}, INV), ({}, {"qdt": ops.BF16}, INV), ({}, {"odt": ops.BF16}, INV),
    ({}, {"ks": FAKE}, INV), ({"kv_dtype": ops.FP8_E4M3}, {}, INV),
    ({"kv_dtype": ops.FP8_E4M3}, {"ks": FAKE, "vs": FAKE, "qdt": ops.F32}, INV),
    ({}, {"q": None}, INV), ({}, {"mask": None}, INV), ({}, {"out": FAKE + 8}, INV), ({}, {"mask": FAKE + 4}, INV),
    ({}, {"ws": None}, INV), ({}, {"wsb": 64}, INV), ({}, {"ws": FAKE + 8}, INV),
    ({}, {"maxb": (1 << 27) + 1}, UNS), ({"num_kv_heads": 1}, {"B": 1 << 20, "maxl": 1 << 20, "maxb": 1 << 16}, UNS),
])
def test_tree_attention_refuses(palib, desc_kw, kw, status):
    assert _tree(_desc(**desc_kw), **kw) == status


def test_tree_workspace_does_not_grow_with_the_batch(palib):
    d = _desc()
    one = palib.pa_tree_attention_workspace_size(4, 64, C.byref(d))   # 128 rows per kv head
    two = palib.pa_tree_attention_workspace_size(4, 65, C.byref(d))
    assert 0 < one < two < 2 * one + 512  # two sets of at most 256 partial rows per CTA
    assert palib.pa_tree_attention_workspace_size(3, 64, C.byref(d)) == 0


def test_accept_and_commit_refuse(palib):
    acc = lambda **kw: palib.pa_tree_accept(*{**dict(d=FAKE, t=FAKE, p=FAKE, qs=FAKE, T=5, B=2, mp=4, path=FAKE,  # noqa: E731
                                                     pl=FAKE, nt=FAKE, st=None), **kw}.values())
    assert acc(B=0) == OK
    for kw in ({"T": -1}, {"B": -1}, {"mp": 0}, {"d": None}, {"qs": None}, {"path": None}, {"nt": FAKE + 4},
               {"d": FAKE + 4}, {"p": FAKE + 2}):
        assert acc(**kw) == INV, kw
    d = _desc()

    def com(desc=d, **kw):
        a = {**dict(k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, mb=4, cl=FAKE, qs=FAKE, path=FAKE, mp=4, pl=FAKE, B=2,
                    nl=FAKE + 64), **kw}
        return palib.pa_tree_commit(*a.values(), C.byref(desc), None)
    assert com(B=0) == OK
    for kw in ({"B": -1}, {"mb": 0}, {"mp": 0}, {"k": None}, {"path": None}, {"ks": FAKE, "vs": FAKE},
               {"nl": FAKE + 4},                      # overlaps context_lens
               {"v": FAKE + 8}, {"pl": FAKE + 2}):
        assert com(**kw) == INV, kw
    assert com(_desc(kv_dtype=ops.INT8)) == INV and com(_desc(block_size=8)) == UNS
    assert com(_desc(num_blocks=(1 << 27) + 5)) == UNS


def test_python_calls_want_cuda_tensors(palib):
    x = torch.zeros(2, 4, 128, dtype=torch.float16)
    kc = torch.zeros(4, 4, 16, 128, dtype=torch.float16)
    i32, i64 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rope_cache_write(x, x, x, i64, torch.ones(64, dtype=torch.float64), i64, kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        ops.tree_attention(x, i32, i64[:, None], kc, kc, i32[None], i32[:1], 16, 2, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        ops.tree_accept(i64, i64, i32, i32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.tree_commit(kc, kc, i32[None], i32[:1], i32[:2], i32[None], i32[:1])


# ---- block manager -----------------------------------------------------------
def test_truncate_releases_trailing_blocks(palib):
    a = ops.BlockAllocator(8)
    a.alloc_seq(1, 40)                       # blocks 0, 1, 2
    slots, _ = a.append_tokens(1, 30)        # 70 tokens: blocks 3, 4
    assert a.table(1) == ([0, 1, 2, 3, 4], 70) and slots[0] == 2 * 16 + 8
    a.truncate_seq(1, 43)
    assert a.table(1) == ([0, 1, 2], 43) and a.free_list() == [5, 6, 7, 3, 4]
    slots, _ = a.append_tokens(1, 1)
    assert slots == [2 * 16 + 11]
    a.fork(1, 2)
    a.truncate_seq(2, 16)                    # shared blocks lose one reference
    assert a.table(1) == ([0, 1, 2], 44) and a.stats()[2][:3] == [2, 1, 1]
    a.truncate_seq(1, 0)
    assert a.table(1) == ([], 0) and a.free_list() == [5, 6, 7, 3, 4, 1, 2]
    for n in (-1, 17):
        with pytest.raises(ops.PagedKVError):
            a.truncate_seq(2, n)
    with pytest.raises(ops.UnknownSequence):
        a.truncate_seq(9, 0)
    assert a.table(2) == ([0], 16)
