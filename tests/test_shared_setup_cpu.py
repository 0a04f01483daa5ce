"""A prefix kernel that cannot run on a device (a build with too few registers for its roles)
is the shared calls' error, and no other call's (read from the sources; no GPU)."""
import os
import re

from paged_kv_decode_06_gb300 import build as builder


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(builder.CSRC, name)).read())


def _body(code, head):
    """A function's text, to the brace that closes it at the line's start."""
    at = code.index(head)
    return code[at:code.index("\n}\n", at)]


def test_the_device_set_up_does_not_fail_for_it():
    body = _body(_code("pa_host.cu"), "int device_state(")
    line = next(x for x in body.splitlines() if "set_shared_smem_limits" in x)
    assert "return" not in line and "s.shared_prefix =" in line and "cudaGetLastError()" in line


def test_the_shared_calls_do():
    code = _code("pa_host_walk.cu")
    assert "dev.shared_prefix != cudaSuccess" in _body(code, "int plan_shared(")
    assert "plan_shared(" in _body(code, "int decode_shared(") and "plan_shared(" in _body(code, "int shared_plan_for(")
    assert "shared_prefix" not in _body(code, "int decode_window(")
