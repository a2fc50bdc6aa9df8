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


def loops(text):
    """The braces' contents of the `for` loops of a text that have braces."""
    for m in re.finditer(r"\bfor \(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        if text[i:].lstrip().startswith("{"):
            yield body(text, i)


@pytest.mark.parametrize("name", ["linear_mma.cu", "moe_mma.cu"])
def test_a_warp_is_whole_again_before_it_reads_tensor_memory(name):
    """tcgen05.ld is for whole warps: the loop that has one and then writes outputs, of which
    lanes may have none or more to do, ends with __syncwarp()."""
    def reads_and_writes(loop):
        at = loop.find("tc_ld_32x32b_x32(")
        return at >= 0 and re.search(r"\bput\(", loop[at:]) is not None

    found = [x for x in loops(source(name)) if reads_and_writes(x)]
    inner = [x for x in found if not any(reads_and_writes(y) for y in loops(x[1:]))]
    assert len(inner) == 1
    assert inner[0][:-1].rstrip().endswith("__syncwarp();"), f"{name}: a loop over tcgen05.ld"


def test_a_warp_is_whole_again_before_the_next_tile():
    text = source("linear_mma.cu")
    ends = [m.end() for m in re.finditer(r"put\(v\[i\], i\);\s*", text)]
    assert ends and all(text[e:].startswith("__syncwarp();") for e in ends)


def test_what_the_lanes_acquired_is_there_for_the_lane_that_copies():
    """Each lane acquires the count of another group and one lane then issues the copies of
    any: only __syncwarp() between orders the one after the others (a vote does not)."""
    text = source("moe_mma.cu")
    look = body(text, text.index("const auto h_ready"))
    assert "load_acquire(" in look and "__ballot_sync(" in look
    last = look.rindex("fence.proxy.async.global")
    assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"$", look[:last])


def test_a_timeout_is_reported_for_waits_and_misplaced_memory_only():
    """kStatusTimeout reaches the caller as MX_ERR_DEVICE_TIMEOUT: in the experts' kernel it
    stands behind the waits' limits and the shared memory's alignment."""
    text = source("moe_mma.cu")
    for m in re.finditer(r"atomicOr\([^;]*kStatusTimeout\)", text):
        before = text[:m.start()].rstrip()
        assert before.endswith("if (!aligned)") or before.endswith("*x.abort = 1u;"), before[-80:]
