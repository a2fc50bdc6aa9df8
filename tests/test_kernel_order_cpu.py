"""Orderings that the kernels' sources have to spell out, because no run shows reliably that
one is missing.  Read from the CUDA sources; no GPU."""
import os
import re

import pytest

from block_scaled_fp4_bf16_gb300 import build as _build

REMOTE = re.compile(r"\b(mapa_shared|st_cluster_f32|ld_cluster_f32x4|bulk_copy_to_cluster)\s*\(")
BARRIER = re.compile(r"\bcluster_(sync|wait)\s*\(\s*\)")


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, at):
    """The braces' content that begins at or after `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def kernels(name):
    text = source(name)
    for m in re.finditer(r"__global__", text):
        yield body(text, m.end())


@pytest.mark.parametrize("name", [s for s in _build.SOURCES if REMOTE.search(source(s))])
def test_a_cluster_has_begun_before_its_shared_memory_is_used(name):
    """A CTA may use another's shared memory only once that one has begun: a barrier of the
    cluster comes before the first such access."""
    found = 0
    for k in kernels(name):
        first = REMOTE.search(k)
        if first is None:
            continue
        found += 1
        assert BARRIER.search(k[:first.start()]), f"{name}: no cluster barrier before {first.group(1)}"
    assert found > 0
