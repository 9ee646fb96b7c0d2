"""Block-scaled caches and sampled verification on the host: the oracle's own
pins and the entry points' refusals.  No GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import scaled as O
from oracle.attention import paged_prefill
from oracle.fp8_e4m3 import e4m3_decode
from paged_kv_cache_191_gb300 import ops, workloads as W
from tests.libfixture import palib  # noqa: F401
from tests.scaled_inputs import Drafts, ScaledBatch
from tests.test_abi import FAKE, _desc

INV, UNS, OK = ops.PA_ERR_INVALID, ops.PA_ERR_UNSUPPORTED, ops.PA_OK


# ---- oracle pins -----------------------------------------------------------
def test_power_scale_is_the_smallest_that_fits():
    for x, want in ((448.0, 1.0), (449.0, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7),
                    (0.0, 0.0), (1e-45, 2.0 ** -126), (3.4e38, 2.0 ** 120)):
        assert O.power_scale([x, -x / 2]) == want
    assert O.power_scale([np.inf, 3.0, np.nan]) == 2.0 ** -7


def test_append_token_by_token_keeps_what_one_call_stores():
    """Codes that stay normal are shifted exactly, so rows stored one at a time
    hold the values that one call rounds to, up to the subnormals' step."""
    w = ScaledBatch(1, 2, 2, [40], [40])
    k, v = w.new_k.numpy(), w.new_v.numpy()
    one = O.append(w.k, w.v, w.k_scale, w.v_scale, k, v, w.q_start, w.tables, w.lens)
    many = [w.k, w.v, w.k_scale, w.v_scale]
    for t in range(40):
        many = O.append(*many, k[t:t + 1], v[t:t + 1], [0, 1], w.tables, [t + 1])
    assert np.array_equal(one[2], many[2]) and np.array_equal(one[3], many[3])
    for c, s, x in ((0, 2, k), (1, 3, v)):
        for g in range(2):
            a, b = O.gather(one[c], one[s], w.tables[0], 40, g), O.gather(many[c], many[s], w.tables[0], 40, g)
            step = np.repeat(one[s][w.tables[0][:3], g], 16)[:40, None] * 2.0 ** -9
            assert (np.abs(a - b) <= step).all()
            assert (np.abs(a - x[:, g]) <= np.abs(x[:, g]) * 2.0 ** -4 + step).all()


def test_a_block_that_starts_afresh_forgets_its_scale():
    w = ScaledBatch(2, 1, 1, [1], [17])
    w.k_scale[:] = 64.0
    out = O.append(w.k, w.v, w.k_scale, w.v_scale, w.new_k.numpy(), w.new_v.numpy(), w.q_start, w.tables, w.lens)
    assert out[2][w.tables[0][1], 0] < 1.0 and out[2][w.tables[0][0], 0] == 64.0
    w.lens[:] = 16  # the last row of the first block: the others stay
    out = O.append(w.k, w.v, w.k_scale, w.v_scale, w.new_k.numpy(), w.new_v.numpy(), w.q_start, w.tables, w.lens)
    assert out[2][w.tables[0][0], 0] == 64.0


def test_attention_is_paged_attention_of_the_values():
    w = ScaledBatch(3, 4, 2, [5, 0, 17], [20, 9, 17])
    got = O.attention(w.q.numpy(), w.q_start, w.k, w.v, w.k_scale, w.v_scale, w.tables, w.lens, w.scale)[0]
    k, v = (e4m3_decode(c) * s.astype(np.float64)[:, :, None, None] for c, s in ((w.k, w.k_scale), (w.v, w.v_scale)))
    want = paged_prefill(w.q.numpy(), w.q_start, k, v, w.tables, w.lens, w.scale)
    assert np.allclose(got, want, rtol=0, atol=1e-12)


def test_verify_by_hand():
    p = np.array([[.5, .3, .2], [.1, .1, .8], [1, 0, 0]], dtype=np.float32)
    q = np.array([[.2, .6, .2], [.1, .1, .8], [0, 1, 0]], dtype=np.float32)
    tok = [0, 1, 2]
    # node 1's token 1: accepted while u * .6 < .3; node 2's token 2: u * .8 < .8
    assert O.verify(tok, p, [.9, .49, .99], [0, 3], 3, draft=q) == ([[0, 1, 2]], [0])
    # refused: what is left of row 0 is token 0's .3
    assert O.verify(tok, p, [.99, .51, .0], [0, 3], 3, draft=q) == ([[0]], [0])
    # without a draft's distribution: u < .3; then token 1 has nothing left
    assert O.verify(tok, p, [.75, .31, .0], [0, 3], 3) == ([[0]], [2])
    assert O.verify(tok, p, [.70, .31, .0], [0, 3], 3) == ([[0]], [0])
    # max_path: drawn from the row of the last accepted node
    assert O.verify(tok, p, [.15, .1, .0], [0, 3], 2) == ([[0, 1]], [1])
    # a tree: the second child has .3 / (1 - .5), the third repeats the first
    assert O.verify([0, 0, 1, 0], np.repeat(p[:1], 4, 0), [.1, .6, .59, .0], [0, 4], 4,
                    parents=[-1, 0, 0, 0]) == ([[0, 2]], [0])
    assert O.verify([0, 0, 1, 0], np.repeat(p[:1], 4, 0), [.1, .6, .61, .0], [0, 4], 4,
                    parents=[-1, 0, 0, 0]) == ([[0]], [2])
    assert O.verify([], p, [], [0, 0], 3) == ([[]], [-1])
    zero = np.zeros((1, 3), dtype=np.float32)
    assert O.verify([0], zero, [.5], [0, 1], 3) == ([[0]], [-1])


def test_draws_compare_whole_sums():
    """u0 times the sum lies 1866 2^-24 below a whole number that is a cumulated sum too, and half of 2^54 - 1 half
    below one: the token there is the first above."""
    m, first, rest = 11191015, 8393261 << 20, 4393167093978
    assert m * (first + rest) == (first << 24) - 1866
    p = np.zeros((2, 1025), dtype=np.float32)
    p[0, :3] = np.array([first, rest >> 20 << 20, rest & 0xFFFFF]) * 2.0 ** -44
    p[1, :1023], p[1, 1023], p[1, 1024] = 1.0, 1.0 - 2.0 ** -24, (2 ** 20 - 1) * 2.0 ** -44
    assert [int(O.fixed(x).sum()) for x in p] == [first + rest, 2 ** 54 - 1]
    assert O.verify([0, 0], p, [m * 2.0 ** -24, 0.5], [0, 1, 2], 2)[1] == [0, 511]


@pytest.mark.parametrize("kind", ["sampled", "picked", "tree"])
def test_verified_tokens_are_distributed_as_the_target(kind):
    """The first token behind node 0, over many draws: each token's share is
    within 5 standard deviations of its probability."""
    rng = W.rng_for(8)
    V, n, runs = 6, 4, 6000
    p = rng.dirichlet(np.ones(V), 1).astype(np.float32).repeat(n, 0)
    q = rng.dirichlet(np.ones(V), 1).astype(np.float32).repeat(n, 0)
    q64 = q[0].astype(np.float64) / q[0].astype(np.float64).sum()
    count = np.zeros(V)
    for _ in range(runs):
        tok = rng.choice(V, n, p=q64) if kind == "sampled" else rng.integers(0, V, n)
        paths, nexts = O.verify(tok, p, rng.random(n, dtype=np.float32), [0, n], n, draft=q if kind == "sampled" else None,
                                parents=[-1, 0, 0, 0] if kind == "tree" else None)
        count[tok[paths[0][1]] if len(paths[0]) > 1 else nexts[0]] += 1
    assert (np.abs(count / runs - p[0]) <= 5 * np.sqrt(p[0] / runs)).all()


# ---- refusals --------------------------------------------------------------
def _d8(**kw):
    return _desc(**{"kv_dtype": ops.FP8_E4M3, **kw})


def _append(d, **kw):
    a = dict(k=FAKE, v=FAKE, dt=ops.F16, ks=256, vs=256, qs=FAKE, T=3, bt=FAKE, mb=4, cl=FAKE, B=2, kc=FAKE, vc=FAKE,
             sk=FAKE, sv=FAKE)
    a.update(kw)
    return ops.lib().pa_block_scaled_append(a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["qs"], a["T"], a["bt"], a["mb"],
                                            a["cl"], a["B"], a["kc"], a["vc"], a["sk"], a["sv"], C.byref(d), None)


@pytest.mark.parametrize("desc_kw,kw,status", [
    ({}, {"k": None}, INV), ({}, {"sk": None}, INV), ({}, {"qs": None}, INV), ({}, {"k": FAKE + 8}, INV),
    ({}, {"sv": FAKE + 2}, INV), ({}, {"dt": ops.FP8_E4M3}, INV), ({}, {"ks": 248}, INV), ({}, {"vs": 260}, INV),
    ({}, {"T": -1}, INV), ({}, {"B": -1}, INV), ({}, {"mb": 0}, INV), ({}, {"mb": 1 << 28}, UNS),
    ({"kv_dtype": ops.INT8}, {}, UNS), ({"kv_dtype": ops.F16}, {}, UNS), ({"head_dim": 64}, {}, UNS),
    ({"block_size": 32}, {}, UNS), ({"num_blocks": 0}, {}, INV), ({}, {"T": 0, "k": None}, OK), ({}, {"B": 0}, OK)])
def test_append_refuses(palib, desc_kw, kw, status):
    assert _append(_d8(**desc_kw), **kw) == status


def _attend(d, **kw):
    a = dict(q=FAKE, dt=ops.F16, st=512, qs=FAKE, T=3, mq=2, kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, bt=FAKE, mb=4, cl=FAKE,
             ml=64, B=2, Hq=4, scale=0.1, out=FAKE, odt=ops.F16, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return ops.lib().pa_block_scaled_attention(
        a["q"], a["dt"], a["st"], a["qs"], a["T"], a["mq"], a["kc"], a["vc"], a["sk"], a["sv"], a["bt"], a["mb"], a["cl"],
        a["ml"], a["B"], a["Hq"], a["scale"], a["out"], a["odt"], C.byref(d), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("desc_kw,kw,status", [
    ({}, {"q": None}, INV), ({}, {"out": FAKE + 4}, INV), ({}, {"sk": None}, INV), ({}, {"sv": FAKE + 1}, INV),
    ({}, {"dt": ops.F32}, INV), ({}, {"odt": ops.BF16}, INV), ({}, {"st": 504}, INV), ({}, {"st": 516}, INV),
    ({}, {"Hq": 3}, INV), ({}, {"Hq": 0}, INV), ({}, {"Hq": 128, "st": 128 * 128}, UNS), ({}, {"mq": 0}, INV),
    ({}, {"mq": 65536}, UNS), ({}, {"scale": float("inf")}, INV), ({}, {"ml": -1}, INV), ({}, {"mb": 0}, INV),
    ({}, {"ws": None}, INV), ({}, {"ws": FAKE + 8}, INV), ({}, {"wsb": 64}, INV), ({"kv_dtype": ops.INT8}, {}, UNS),
    ({"head_dim": 64}, {}, UNS), ({}, {"T": 1 << 30, "ml": 1 << 20}, UNS), ({}, {"T": 0, "q": None, "ws": None}, OK),
    ({}, {"B": 0, "ws": None}, OK)])
def test_attention_refuses(palib, desc_kw, kw, status):
    assert _attend(_d8(**desc_kw), **kw) == status


def test_attention_workspace_size(palib):
    size = palib.pa_block_scaled_attention_workspace_size
    assert 0 < size(4, 1, C.byref(_d8())) < size(4, 8, C.byref(_d8())) < size(4, 100, C.byref(_d8()))
    assert size(4, 100, C.byref(_d8())) == size(4, 60000, C.byref(_d8()))
    assert size(3, 1, C.byref(_d8())) == size(4, 1, C.byref(_desc())) == size(4, -1, C.byref(_d8())) == 0


def test_items_below_128_rows_hold_a_whole_sequence(palib):
    """What the planner of the thread-per-key kernels relies on.  The rows of an item come out of the workspace: two
    sets of rows of D + 2 floats a CTA, and 32 bytes."""
    size = palib.pa_block_scaled_attention_workspace_size
    sms = next(n for n in range(1, 1000) if abs(size(1, 1, C.byref(_d8(num_kv_heads=1))) - n * (2 * 8 * 130 * 4 + 32)) < 256)
    for G in range(1, 33):
        heads = 1 << (G - 1).bit_length()
        for n in range(1, 200):
            rows = round((size(G, n, C.byref(_d8(num_kv_heads=1))) / sms - 32) / (2 * 130 * 4))
            assert rows == 128 or (rows in (8, 16, 32, 40) and heads * n <= rows and rows % heads == 0)


def _copy(d, **kw):
    a = dict(dk=FAKE, dv=FAKE, dks=FAKE, dvs=FAKE, dn=8, sk=FAKE, sv=FAKE, sks=FAKE, svs=FAKE, sn=8, p=FAKE, n=2)
    a.update(kw)
    return ops.lib().pa_block_scaled_copy(a["dk"], a["dv"], a["dks"], a["dvs"], a["dn"], a["sk"], a["sv"], a["sks"],
                                          a["svs"], a["sn"], a["p"], a["n"], C.byref(d), None)


@pytest.mark.parametrize("desc_kw,kw,status", [
    ({}, {"dk": None}, INV), ({}, {"svs": None}, INV), ({}, {"p": FAKE + 4}, INV), ({}, {"n": -1}, INV),
    ({}, {"dn": 0}, INV), ({}, {"sn": -3}, INV), ({"kv_dtype": ops.BF16}, {}, UNS), ({}, {"n": 0, "p": None}, OK)])
def test_copy_refuses(palib, desc_kw, kw, status):
    assert _copy(_d8(**desc_kw), **kw) == status


def _verify(**kw):
    a = dict(t=FAKE, p=FAKE, ps=100, q=None, qst=0, V=100, u=FAKE, par=None, qs=FAKE, T=4, B=2, mp=3, path=FAKE,
             pl=FAKE, nt=FAKE)
    a.update(kw)
    return ops.lib().pa_draft_verify(a["t"], a["p"], a["ps"], a["q"], a["qst"], a["V"], a["u"], a["par"], a["qs"], a["T"],
                                     a["B"], a["mp"], a["path"], a["pl"], a["nt"], None)


@pytest.mark.parametrize("kw,status", [
    ({"t": None}, INV), ({"p": None}, INV), ({"u": None}, INV), ({"qs": None}, INV), ({"path": None}, INV),
    ({"nt": None}, INV), ({"t": FAKE + 4}, INV), ({"p": FAKE + 2}, INV), ({"V": 0}, INV), ({"ps": 99}, INV),
    ({"q": FAKE, "qst": 99}, INV), ({"V": (1 << 19) + 1, "ps": 1 << 20}, UNS),
    ({"q": FAKE, "qst": 100, "par": FAKE}, UNS), ({"mp": 0}, INV), ({"T": -1}, INV), ({"B": -1}, INV),
    ({"B": 0, "path": None}, OK)])
def test_verify_refuses(palib, kw, status):
    assert _verify(**kw) == status


def test_wrappers_want_cuda_tensors():
    w = ScaledBatch(4, 2, 2, [1], [5])
    t = torch.from_numpy
    cache = [t(w.k), t(w.v), t(w.k_scale), t(w.v_scale)]
    with pytest.raises(ValueError):
        ops.block_scaled_append(w.new_k, w.new_v, t(w.q_start), t(w.tables), t(w.lens), *cache)
    with pytest.raises(ValueError):
        ops.block_scaled_attention(w.q, t(w.q_start), *cache, t(w.tables), t(w.lens), 5, 1, 0.1)
    with pytest.raises(ValueError):
        ops.block_scaled_copy(*cache, *cache, torch.zeros((0, 2), dtype=torch.int64))
    d = Drafts(1, [2], 5, "sampled")
    with pytest.raises(ValueError):
        ops.draft_verify(t(d.tokens), t(d.target), t(d.uniform), t(d.q_start), 2)
