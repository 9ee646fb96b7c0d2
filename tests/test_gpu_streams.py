"""Calls given a stream that is not the current one: scratch and results that
the call allocates belong to that stream, and the results are those of the call
on the current stream."""
import numpy as np
import pytest
import torch

from paged_kv_cache_191_gb300 import ops, workloads as W
from tests.gpu_util import held_by_a_call_on_another_stream, requires_cuda
from tests.test_gpu_decode_grouped import grouped_case, last_slots

pytestmark = [pytest.mark.gpu, requires_cuda]
DEV = "cuda"


@pytest.mark.parametrize("what", ["decode", "chunked_prefill", "decode_append", "grouped", "segments"])
def test_a_call_keeps_its_memory_on_another_stream(monkeypatch, what):
    w, start = grouped_case(51, [4, 2], [40, 12], 4, 2, "f16")
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    q, k, v = (t.to(DEV) for t in (w.q, w.k_pool, w.v_pool))
    tables, lens = on(w.block_tables.astype(np.int32)), on(w.context_lens.astype(np.int32))
    most, slots = int(w.context_lens.max()), on(last_slots(w))
    rng = W.rng_for(3)
    new = [W.randn(rng, (w.B, 2, 128), torch.float16).to(DEV) for _ in range(2)]
    common = (q, k, v, tables, lens, most, w.scale)
    items, most_items = ops.shared_table_segments(w.block_tables, w.context_lens, start)
    # 40 query tokens of the first sequence, one of each other
    starts = on(np.concatenate([[0], 40 + np.arange(w.B)]).astype(np.int32))
    qt = W.randn(rng, (39 + w.B, 4, 128), torch.float16).to(DEV)
    gs, prefix, items = on(start), on(np.array([40, 12], np.int32)), on(items)
    call = {"decode": lambda s: [ops.decode(*common, split_tokens=128, stream=s)],
            "chunked_prefill": lambda s: [ops.chunked_prefill(qt, starts, k, v, tables, lens, most, 40, w.scale,
                                                              split_tokens=128, stream=s)],
            "decode_append": lambda s: [ops.decode_append(*new, slots, *common, split_tokens=128, stream=s)],
            "grouped": lambda s: [ops.decode_append_grouped(*new, slots, *common, gs, prefix, 4, 40, split_tokens=128,
                                                            stream=s)],
            "segments": lambda s: [ops.decode_append_segments(*new, slots, *common, gs, items, 4, most_items,
                                                              stream=s)]}[what]
    ops.device_errors(clear=True)
    plain, other = held_by_a_call_on_another_stream(monkeypatch, ops, call)
    assert ops.device_errors(clear=True) == 0
    assert all(torch.equal(x, y) for x, y in zip(plain, other))
