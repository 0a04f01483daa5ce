"""A kernel that gives up on a wait ends behind its own copies and products: each source
that issues some waits for the last of them, with a limit that no call sets (read from
the sources; no GPU)."""
import os
import re

import pytest

from paged_kv_decode_06_gb300 import build as builder

KERNELS = {
    # source: (waits for copies, waits for products) of the last phases
    "pa_split.cuh": (2, 0),
    "pa_shared.cu": (1, 1),
}


def _code(name):
    text = open(os.path.join(builder.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", list(KERNELS))
def test_the_last_copies_and_products_are_waited_for(name):
    code = _code(name)
    waits = re.findall(r"\w*wait\(([^;]*?)kDrainNs\)", code, flags=re.S)
    assert len(waits) == sum(KERNELS[name])
    assert sum("drain" in w for w in waits) == KERNELS[name][1]
    # no other limit than the call's beside it
    assert not re.findall(r"drain\w*(?:\(\w+\))?, 0u, p\.wait_ns", code)
