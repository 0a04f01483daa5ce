"""The kernels of a shared call that do not wait for the grid before them: what they read of
it stands behind an acquire of the plan's release (read from the sources; no GPU)."""
import os
import re

from paged_kv_decode_06_gb300 import build as builder


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(builder.CSRC, name)).read())


def test_the_split_kernel_acquires_the_plan():
    code = _code("pa_split.cuh")
    body = code[code.index("pa_split_kernel("):]
    own = body[body.index("if constexpr (WALK == Walk::kOwn)"):]
    own = own[:own.index("return;")]
    assert "load_acquire(p.ready)" in own and "grid_dependency_wait()" in own
    # nothing of global memory before it
    before = body[:body.index("load_acquire(p.ready)")]
    assert not re.search(r"__ldcg|p\.(skip|qsl|seq_lens|block_tables)\b", before)


def test_the_plan_releases_last_and_the_merge_takes_the_word_back():
    plan = _code("pa_shared.cu")
    plan = plan[plan.index("pa_shared_plan_kernel("):]
    plan = plan[:plan.index("\n}\n")]
    tail = plan[plan.index("store_release(p.ready"):]
    assert "p." not in tail[tail.index(";"):] and plan.rindex("__syncthreads()") > plan.rindex("p.skip[")
    merge = _code("pa_merge_rows.cu")
    assert merge.index("grid_dependency_wait()") < merge.index("*p.ready = 0")
