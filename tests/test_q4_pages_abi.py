"""Host checks of the 4-bit cache's and the page operations' entry points: what
they refuse before anything reaches the device (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import build as builder

BAD, UNS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED


@pytest.fixture(autouse=True)
def _no_gpu():
    """These calls pass host tensors: where a GPU is present a call that the checks let
    through would run on their memory."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.load()


def _passes(st):
    """Every host check passed: without a GPU the call then fails at device set-up."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert st == binding.PA_ERR_CUDA, binding.paged_attn_last_error_message()


def _refs(*tensors, fp4=()):
    d = [binding.tensor_desc(t, binding._fp4_code) if i in fp4 else binding.tensor_desc(t)
         for i, t in enumerate(tensors)]
    return [ctypes.byref(x) for x in d]


# --------------------------------------------------------------------- rows

def _rows(T=4, Hkv=2, D=64, NB=3):
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    return dict(key=torch.zeros(T, Hkv, D, dtype=torch.bfloat16), value=torch.zeros(T, Hkv, D, dtype=torch.bfloat16),
                slots=torch.zeros(T, dtype=torch.int32), kc=z(NB, 16, Hkv, D // 2), vc=z(NB, 16, Hkv, D // 2),
                ks=z(NB, Hkv, 16, D // 16), vs=z(NB, Hkv, 16, D // 16))


def _write(lib, a, s=1.0):
    r = _refs(a["key"], a["value"], a["slots"], a["kc"], a["vc"], a["ks"], a["vs"], fp4=(3, 4))
    return lib.paged_attn_cache_write_q4(*r, s, 1.0, None)


def _read(lib, a, s=1.0):
    r = _refs(a["slots"], a["kc"], a["vc"], a["ks"], a["vs"], a["key"], a["value"], fp4=(1, 2))
    return lib.paged_attn_cache_read_q4(*r[:5], 1.0, s, *r[5:], None)


def test_valid_rows_pass(lib):
    _passes(_write(lib, _rows()))
    _passes(_read(lib, _rows(T=1, Hkv=3, D=16)))


def test_no_rows_is_nothing_to_do(lib):
    assert _write(lib, _rows(T=0)) == binding.PA_OK
    assert _read(lib, _rows(T=0)) == binding.PA_OK


@pytest.mark.parametrize("mutate,expect", [
    (lambda a: a.update(key=a["key"].float()), BAD),
    (lambda a: a.update(value=torch.zeros(4, 2, 32, dtype=torch.bfloat16)), BAD),
    (lambda a: a.update(slots=a["slots"].long()), BAD),
    (lambda a: a.update(slots=torch.zeros(3, dtype=torch.int32)), BAD),
    (lambda a: a.update(slots=torch.zeros(8, dtype=torch.int32)[::2]), BAD),
    (lambda a: a.update(kc=a["kc"].to(torch.int32)), BAD),
    (lambda a: a.update(kc=torch.zeros(3, 8, 2, 32, dtype=torch.uint8)), UNS),
    (lambda a: a.update(vc=torch.zeros(3, 16, 2, 64, dtype=torch.uint8)), BAD),
    (lambda a: a.update(vc=torch.zeros(4, 16, 2, 32, dtype=torch.uint8)), BAD),
    (lambda a: a.update(kc=torch.zeros(3, 16, 2, 36, dtype=torch.uint8)[..., :32]), BAD),      # stride 36
    (lambda a: a.update(kc=torch.zeros(3, 16, 2, 40, dtype=torch.uint8)[..., 4:36]), BAD),     # address
    (lambda a: a.update(ks=torch.zeros(3, 2, 16, 8, dtype=torch.uint8)), BAD),
    (lambda a: a.update(vs=torch.zeros(3, 16, 2, 4, dtype=torch.uint8)), BAD),
    (lambda a: a.update(vs=a["vs"].float()), BAD),
    (lambda a: a.update(vs=None), BAD),
    (lambda a: a.update(key=torch.zeros(4, 2, 66, dtype=torch.bfloat16)[..., :64]), BAD),
])
def test_rows_refused(lib, mutate, expect):
    for call in (_write, _read):
        a = _rows()
        mutate(a)
        assert call(lib, a) == expect, binding.paged_attn_last_error_message()
        assert binding.paged_attn_last_error_message() != ""


@pytest.mark.parametrize("D", [8, 24, 528])
def test_head_dims_outside_the_envelope(lib, D):
    a = _rows(D=16)
    a.update(key=torch.zeros(4, 2, D, dtype=torch.bfloat16), value=torch.zeros(4, 2, D, dtype=torch.bfloat16))
    assert _write(lib, a) == UNS and _read(lib, a) == UNS


@pytest.mark.parametrize("s", [0.0, -1.0, float("nan"), float("inf")])
def test_tensor_scales_must_be_positive(lib, s):
    assert _write(lib, _rows(), s) == BAD and _read(lib, _rows(), s) == BAD


def test_broadcast_destinations_are_refused(lib):
    a = _rows()
    a["kc"] = torch.zeros(1, 16, 2, 32, dtype=torch.uint8).expand(3, 16, 2, 32)
    assert _write(lib, a) == BAD
    _passes(_read(lib, a))                         # read only: fine
    a = _rows()
    a["key"] = torch.zeros(4, 1, 64, dtype=torch.bfloat16).expand(4, 2, 64)
    assert _read(lib, a) == BAD
    _passes(_write(lib, a))


# ------------------------------------------------------------------- decode

def _decode_args(T=3, B=3, Hq=8, Hkv=2, D=64, NB=5, MB=4):
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(q=torch.zeros(T, Hq, D, dtype=torch.bfloat16), kc=z(NB, 16, Hkv, D // 2), vc=z(NB, 16, Hkv, D // 2),
                ks=z(NB, Hkv, 16, D // 16), vs=z(NB, Hkv, 16, D // 16), bt=i(B, MB), sl=i(B), qsl=None,
                out=torch.zeros(T, Hq, D, dtype=torch.bfloat16), lse=torch.zeros(T, Hq), runs=1, scale=0.1, ks1=1.0,
                vs1=1.0, opts=None, fp4=(1, 2))


def _decode(lib, a):
    r = _refs(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["qsl"], a["out"], a["lse"], fp4=a["fp4"])
    o = binding.make_options(**a["opts"]) if a["opts"] else None
    return lib.paged_attn_decode_q4(*r[:8], a["runs"], a["scale"], a["ks1"], a["vs1"], *r[8:],
                                    ctypes.byref(o) if o is not None else None, None)


def test_valid_decodes_pass(lib):
    _passes(_decode(lib, _decode_args()))
    a = _decode_args(T=5, B=2, Hq=16, Hkv=16, D=128)
    _passes(_decode(lib, dict(a, qsl=torch.zeros(3, dtype=torch.int32), runs=4, lse=None, opts=dict(heads_per_cta=4))))


def test_no_query_tokens_is_nothing_to_do(lib):
    assert _decode(lib, _decode_args(T=0, B=0)) == binding.PA_OK


@pytest.mark.parametrize("change,expect", [
    (dict(q=torch.zeros(3, 8, 64)), BAD),                                              # not bf16
    (dict(q=torch.zeros(3, 7, 64, dtype=torch.bfloat16)), BAD),                        # heads not a multiple
    (dict(q=torch.zeros(3, 8, 128, dtype=torch.bfloat16)), BAD),                       # other head size than the codes'
    (dict(q=torch.zeros(3, 8, 66, dtype=torch.bfloat16)[:, :, :64]), BAD),             # heads apart
    (dict(q=torch.zeros(3 * 8 * 64 + 1, dtype=torch.bfloat16)[1:].view(3, 8, 64)), BAD),   # 2-byte aligned
    (dict(fp4=()), BAD),                                                               # bytes, not codes
    (dict(kc=torch.zeros(5, 32, 2, 32, dtype=torch.uint8)), UNS),                      # page size
    (dict(vc=torch.zeros(4, 16, 2, 32, dtype=torch.uint8)), BAD),                      # fewer pages
    (dict(vc=torch.zeros(5, 16, 2, 40, dtype=torch.uint8)[:, :, :, :32]), BAD),        # strides of 40 bytes
    (dict(kc=torch.zeros(5, 16, 2, 64, dtype=torch.uint8)[:, :, :, ::2]), BAD),
    (dict(ks=torch.zeros(5, 16, 2, 4, dtype=torch.uint8).transpose(1, 2)), BAD),       # a page's scales not contiguous
    (dict(vs=torch.zeros(5, 2, 16, 3, dtype=torch.uint8)), BAD),
    (dict(ks=torch.zeros(5, 2, 16, 4)), BAD),
    (dict(bt=torch.zeros(3, 4, dtype=torch.int64)), BAD),
    (dict(bt=torch.zeros(4, 3, dtype=torch.int32).t()), BAD),
    (dict(bt=torch.zeros(1, dtype=torch.int32).expand(3, (1 << 27) - 63)), UNS),       # 2^31 tokens
    (dict(sl=torch.zeros(2, dtype=torch.int32)), BAD),
    (dict(qsl=torch.zeros(3, dtype=torch.int32)), BAD),
    (dict(runs=2), BAD),                                                               # runs without offsets
    (dict(runs=0), BAD),
    (dict(qsl=torch.zeros(4, dtype=torch.int32), runs=17), UNS),                       # 4 x 17 rows
    (dict(out=torch.zeros(3, 8, 32, dtype=torch.bfloat16)), BAD),
    (dict(out=torch.zeros(1, 8, 64, dtype=torch.bfloat16).expand(3, 8, 64)), BAD),
    (dict(lse=torch.zeros(3, 4)), BAD),
    (dict(lse=torch.zeros(1, 1).expand(3, 8)), BAD),
    (dict(scale=float("nan")), BAD),
    (dict(ks1=float("inf")), BAD),
    (dict(opts=dict(heads_per_cta=3)), BAD),
    (dict(opts=dict(num_ctas=1 << 15)), BAD),
    (dict(opts=dict(num_ctas=-1)), BAD),
    (dict(opts=dict(page_pairing=1)), UNS),
])
def test_decodes_refused(lib, change, expect):
    st = _decode(lib, dict(_decode_args(), **change))
    assert st == expect, (st, binding.paged_attn_last_error_message())


def test_decode_pages_far_apart_are_refused(lib):
    a = _decode_args(NB=1)
    d = binding._new_desc(a["kc"], binding._fp4_code)
    d.stride[0] = 1 << 32
    r = _refs(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], None, a["out"], a["lse"], fp4=(1, 2))
    r[1] = ctypes.byref(d)
    assert lib.paged_attn_decode_q4(*r[:8], 1, 0.1, 1.0, 1.0, *r[8:], None, None) == UNS


# -------------------------------------------------------------------- pages

def _array(tensors):
    return (binding.PaTensor * max(1, len(tensors)))(*[binding.tensor_desc(t, binding._bytes_code) for t in tensors])


def _i(*x):
    return torch.tensor(x, dtype=torch.int32)


def _page(NB=6):
    return dict(caches=[torch.zeros(NB, 16, 2, 32, dtype=torch.uint8)], bt=torch.zeros(3, 4, dtype=torch.int32),
                sl=_i(0, 0, 0), ref=torch.zeros(NB, dtype=torch.int32), a=_i(0, 1), b=_i(2, 3), c=_i(4, 5),
                all=torch.zeros(NB, dtype=torch.int32), one=_i(0), n=None)


def _n(a):
    return len(a["caches"]) if a["n"] is None else a["n"]


def _copy(lib, a):
    return lib.paged_attn_pages_copy(_array(a["caches"]), _n(a), *_refs(a["a"], a["b"]), None)


def _fork(lib, a):
    return lib.paged_attn_pages_fork(_array(a["caches"]), _n(a),
                                     *_refs(a["bt"], a["sl"], a["ref"], a["a"], a["b"], a["c"]), None)


def _free(lib, a):
    return lib.paged_attn_pages_free(*_refs(a["bt"], a["sl"], a["ref"], a["a"], a["all"], a["one"]), None)


def _compact(lib, a):
    return lib.paged_attn_pages_compact(_array(a["caches"]), _n(a),
                                        *_refs(a["bt"], a["ref"], a["all"], a["one"]), None)


@pytest.mark.parametrize("call", [_copy, _fork, _free, _compact])
def test_valid_page_calls_pass(lib, call):
    _passes(call(lib, _page()))


def test_no_entries_is_nothing_to_do(lib):
    a = _page()
    a.update(a=_i(), b=_i(), c=_i())
    assert _copy(lib, a) == binding.PA_OK and _fork(lib, a) == binding.PA_OK
    a["caches"] = []
    assert _copy(lib, a) == BAD                    # a copy of nothing has no pool
    _passes(_compact(lib, a))                      # tables and counts alone


@pytest.mark.parametrize("mutate,expect", [
    (lambda a: a.update(caches=[torch.zeros(5, 16, 2, 32, dtype=torch.uint8), a["caches"][0]]), BAD),
    (lambda a: a.update(caches=[torch.zeros(6, 8, dtype=torch.float64)]), BAD),
    (lambda a: a.update(caches=[torch.zeros(6, dtype=torch.uint8)]), BAD),
    (lambda a: a.update(caches=[torch.zeros(6, 1, 8, dtype=torch.uint8).expand(6, 4, 8)]), BAD),
    (lambda a: a.update(caches=[torch.zeros(6, 7, 8, 9, dtype=torch.uint8)[:, ::2, ::2, ::2]]), UNS),
    (lambda a: a.update(caches=[torch.zeros(6, 4, 0, dtype=torch.uint8)]), BAD),
    (lambda a: a.update(n=-1), None),
    (lambda a: a.update(n=1025), UNS),
])
def test_caches_refused(lib, mutate, expect):
    for call in (_copy, _fork, _compact):
        a = _page()
        mutate(a)
        st = call(lib, a)
        assert st == expect if expect is not None else st in (BAD, UNS), binding.paged_attn_last_error_message()
        assert binding.paged_attn_last_error_message() != ""


@pytest.mark.parametrize("call,mutate", [
    (_copy, lambda a: a.update(b=_i(1))),
    (_copy, lambda a: a.update(a=a["a"].long())),
    (_copy, lambda a: a.update(a=_i(1, 2, 3, 4)[::2])),
    (_fork, lambda a: a.update(b=_i(1))),
    (_fork, lambda a: a.update(c=a["c"].float())),
    (_fork, lambda a: a.update(sl=_i(0, 0))),
    (_fork, lambda a: a.update(bt=a["bt"].long())),
    (_fork, lambda a: a.update(bt=torch.zeros(4, 3, dtype=torch.int32).t())),
    (_fork, lambda a: a.update(bt=torch.zeros(1, 4, dtype=torch.int32).expand(3, 4))),
    (_fork, lambda a: a.update(ref=torch.zeros(7, dtype=torch.int32))),
    (_free, lambda a: a.update(all=torch.zeros(5, dtype=torch.int32))),
    (_free, lambda a: a.update(one=_i(0, 0))),
    (_free, lambda a: a.update(one=None)),
    (_free, lambda a: a.update(sl=None)),
    (_free, lambda a: a.update(ref=torch.zeros(6, 1, dtype=torch.int32))),
    (_compact, lambda a: a.update(all=torch.zeros(7, dtype=torch.int32))),
    (_compact, lambda a: a.update(one=torch.zeros(1))),
    (_compact, lambda a: a.update(bt=None)),
])
def test_lists_and_tables_refused(lib, call, mutate):
    a = _page()
    mutate(a)
    assert call(lib, a) == BAD, binding.paged_attn_last_error_message()
    assert binding.paged_attn_last_error_message() != ""


def test_null_pointers(lib):
    a = _page()
    r = _refs(a["a"], a["b"])
    assert lib.paged_attn_pages_copy(None, 1, *r, None) == BAD
    assert lib.paged_attn_pages_copy(_array(a["caches"]), 1, None, r[1], None) == BAD
    assert lib.paged_attn_pages_free(*[None] * 6, None) == BAD


def test_binding_refuses_host_tensors():
    a = _page()
    with pytest.raises(ValueError):
        binding.paged_attn_pages_copy(a["caches"], a["a"], a["b"])
    with pytest.raises(ValueError):
        binding.paged_attn_pages_free(a["bt"], a["sl"], a["ref"], a["a"])
