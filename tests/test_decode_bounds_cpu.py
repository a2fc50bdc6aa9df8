"""The bounds-checked build's checks in the decoding step's sources: each plain access to global memory by an
index stands behind in_bounds.  Read from the sources; no GPU."""
import re

import pytest

from tests.test_kernel_order_cpu import source

# the arrays in global memory that the kernels reach by an index
ARRAYS = {
    "kv_cache.cuh": r"\bc\.(lengths|table)\[",
    "kv_append.cu": r"\b(a\.starts|c\.lengths|c\.table)\[|(?<!uint8_t )\*scale\b|\+ at\) =|a\.x\[which\] \+ at",
    "attention.cu": r"\b(a\.lse|plan\.splits|c\.table|c\.lengths|c\.scales\[[01]\])\[|\.state\[|\bp\.sums \+|\ba\.(out|q) \+",
    "qk_rope.cu": r"\b(a\.inv_freq|a\.partials|a\.positions|weight|out)\[|\(p \+ to\)",
    "sample.cu": r"\b(a\.top_p|a\.top_k|a\.temperature|a\.ids|a\.probability|p)\[(row|i)\]|\(a\.logits\)(\[| \+ e)",
}


def guarded(text, at):
    """Is there a check in the access's own statement, in an `if` around it, or shortly before it as one that
    leaves (`if (!in_bounds(..)) return`)?"""
    own = max(text.rfind(c, 0, at) for c in ";{}")
    if "in_bounds(" in text[own:at]:
        return True
    near = own
    for _ in range(6):
        near = max(text.rfind(";", 0, near), 0)
    if re.search(r"if \(!in_bounds\([^;]*\)\) (return|continue)", text[near:at]):
        return True
    depth = 0
    for i in range(at - 1, -1, -1):  # the headers of the braces around it
        depth += {"}": 1, "{": -1}.get(text[i], 0)
        if depth < 0:
            depth = 0
            header = text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i]
            if "in_bounds(" in header:
                return True
            if "__global__" in header or "__device__" in header:
                return False
    return False


@pytest.mark.parametrize("name", list(ARRAYS))
def test_accesses_ask_first(name):
    text = source(name)
    found = list(re.finditer(ARRAYS[name], text))
    assert found
    bad = [text[max(0, m.start() - 60):m.end() + 20] for m in found if not guarded(text, m.start())]
    assert not bad, "\n---\n".join(bad)
