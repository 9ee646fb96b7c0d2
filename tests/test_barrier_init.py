"""Barriers in shared memory: the thread that initialises them makes that visible to
the asynchronous proxy (copies and products that arrive on them) by its own fence.
Checked in the sources: no call makes a missing fence show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_191_gb300", "csrc")
FILES = sorted(f for f in glob.glob(os.path.join(CSRC, "*.cu*")) if "mbar_init(" in open(f, encoding="utf-8").read()
               and not f.endswith("device_common.cuh"))


def enclosing(text, at):
    """The blocks around a place, from the inside out: (what stands before the brace, the block)."""
    depth, i = 0, at
    while i > 0:
        i -= 1
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
                continue
            end, d = i, 0
            while True:
                d += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if d == 0:
                    break
            head = text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i]
            yield head, text[i:end]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_who_initialises_barriers_fences(path):
    text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
    calls = [m.start() for m in re.finditer(r"mbar_init\(", text)]
    assert calls
    for at in calls:
        block = next(b for head, b in enclosing(text, at) if re.search(r"if \((threadIdx\.x|lane|tid|wid)\b", head))
        assert "fence_barrier_init()" in block[block.rindex("mbar_init("):], text[at:at + 60]
