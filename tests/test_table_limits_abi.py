"""Block tables whose rows could hold 2^31 pages in all are refused: the decode
kernels number a batch's pages in int32 (host checks, no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import build as builder


@pytest.fixture(autouse=True)
def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: calls that pass the checks would run on host memory")


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.load()


def _table(rows, cols):
    """Descriptor of an int32 table of that size whose rows share memory."""
    d = binding._new_desc(torch.zeros(2, 2, dtype=torch.int32))
    d.shape[0], d.shape[1], d.stride[0], d.stride[1] = rows, cols, 0, 1
    return d


def _call(lib, kind, rows, cols):
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    sl, lse = torch.ones(rows, dtype=torch.int32), torch.zeros(rows, 8 if kind != "mla" else 16)
    if kind == "q4":
        q, code, sc = b16(rows, 8, 64), u8(3, 16, 2, 32), u8(3, 2, 16, 4)
        c = [binding._new_desc(code, binding._fp4_code)] * 2 + [binding._new_desc(sc)] * 2
        fn, scales = lib.paged_attn_decode_q4, (0.1, 1.0, 1.0)
    elif kind == "bf16":
        q, c = b16(rows, 8, 64), [binding._new_desc(b16(3, 16, 2, 64))] * 2
        fn, scales = lib.paged_attn_decode, (0.1, 1.0, 1.0)
    else:
        q, c = b16(rows, 16, 576), [binding._new_desc(b16(3, 16, 576))]
        fn, scales = lib.paged_attn_mla_decode, (0.1, 1.0)
    out = torch.zeros_like(q) if kind != "mla" else b16(rows, 16, 512)
    d = [binding._new_desc(q), *c, _table(rows, cols), binding._new_desc(sl), binding._new_desc(None)]
    tail = [binding._new_desc(out), binding._new_desc(lse)]
    args = [*map(ctypes.byref, d), 1, *scales, *map(ctypes.byref, tail)]
    return fn(*args, None, None) if kind == "q4" else fn(*args, None)


@pytest.mark.parametrize("kind", ["q4", "bf16", "mla"])
def test_tables_of_two_to_the_31_pages_are_refused(lib, kind):
    assert _call(lib, kind, 32, 1 << 26) == binding.PA_ERR_UNSUPPORTED
    st = _call(lib, kind, 32, (1 << 26) - 1)
    assert st == binding.PA_ERR_CUDA, binding.paged_attn_last_error_message()      # past the checks: no device here
