"""Host checks of paged_attn_rope_cache_write: what it refuses before anything
reaches the device (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import build as builder

BAD, UNS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED
bf = torch.bfloat16


@pytest.fixture(autouse=True)
def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.load()


def _args(T=4, Hq=4, Hkv=2, D=64, NB=3, R=32, P=10, axes=2, kv=bf):
    return dict(q=torch.zeros(T, Hq, D, dtype=bf), k=torch.zeros(T, Hkv, D, dtype=bf),
                v=torch.zeros(T, Hkv, D, dtype=bf), pos=torch.zeros(axes, T, dtype=torch.int32),
                tab=torch.zeros(P, R), axis=bytes([0] * (R // 4) + [axes - 1] * (R // 4)), sl=torch.zeros(T, dtype=torch.int32),
                kc=torch.zeros(NB, 16, Hkv, D, dtype=kv), vc=torch.zeros(NB, 16, Hkv, D, dtype=kv), ks=1.0, vs=1.0,
                qo=torch.zeros(T, Hq, D, dtype=bf), ko=None)


def _call(lib, a):
    d = {n: binding.tensor_desc(a[n]) for n in ("q", "k", "v", "pos", "tab", "sl", "kc", "vc", "qo", "ko")}
    r = {n: ctypes.byref(x) for n, x in d.items()}
    return lib.paged_attn_rope_cache_write(r["q"], r["k"], r["v"], r["pos"], r["tab"], a["axis"], 0, r["sl"], r["kc"],
                                           r["vc"], a["ks"], a["vs"], r["qo"], r["ko"], None)


@pytest.mark.parametrize("make", [
    lambda: _args(), lambda: _args(kv=torch.uint8), lambda: _args(D=40, R=12, axes=3), lambda: dict(_args(), axis=None),
    lambda: dict(_args(axes=1), pos=torch.zeros(4, dtype=torch.int32)),
    lambda: dict(_args(), ko=torch.zeros(4, 2, 64, dtype=bf)),
    lambda: dict(_args(D=512, R=512)), lambda: dict(_args(T=1), q=torch.zeros(1, 4, 64, dtype=bf))])
def test_valid_calls_pass(lib, make):
    # every host check passed: without a GPU the call then fails at device set-up
    assert _call(lib, make()) == binding.PA_ERR_CUDA, binding.paged_attn_last_error_message()


def test_no_tokens_is_no_work(lib):
    assert _call(lib, _args(T=0)) == binding.PA_OK


@pytest.mark.parametrize("change,want", [
    (dict(q=torch.zeros(4, 4, 64)), BAD), (dict(v=torch.zeros(4, 1, 64, dtype=bf)), BAD),
    (dict(k=torch.zeros(5, 2, 64, dtype=bf)), BAD), (dict(pos=torch.zeros(2, 4)), BAD),
    (dict(pos=torch.zeros(2, 5, dtype=torch.int32)), BAD), (dict(pos=torch.zeros(4, 4, dtype=torch.int32)), UNS),
    (dict(pos=torch.zeros(4, 2, dtype=torch.int32).t()), BAD), (dict(tab=torch.zeros(10, 32, dtype=bf)), BAD),
    (dict(tab=torch.zeros(10, 30), axis=bytes(15)), UNS), (dict(tab=torch.zeros(10, 68), axis=bytes(34)), BAD),
    (dict(tab=torch.zeros(10, 34)[:, :32]), BAD), (dict(tab=torch.zeros(1, 32).expand(10, 32)), BAD),
    (dict(tab=torch.zeros(32, 12).t()), BAD), (dict(axis=bytes([2] * 16)), BAD), (dict(sl=torch.zeros(3, dtype=torch.int32)), BAD),
    (dict(sl=torch.zeros(4, dtype=torch.int64)), BAD), (dict(kc=torch.zeros(3, 16, 2, 64)), BAD),
    (dict(kc=torch.zeros(3, 16, 2, 64, dtype=torch.uint8)), BAD),
    (dict(kc=torch.zeros(3, 8, 2, 64, dtype=bf), vc=torch.zeros(3, 8, 2, 64, dtype=bf)), UNS),
    (dict(kc=torch.zeros(3, 16, 1, 64, dtype=bf)), BAD), (dict(vc=torch.zeros(4, 16, 2, 64, dtype=bf)), BAD),
    (dict(vc=torch.zeros(1, 16, 2, 64, dtype=bf).expand(3, 16, 2, 64)), BAD),
    (dict(qo=torch.zeros(4, 4, 64)), BAD), (dict(qo=torch.zeros(4, 2, 64, dtype=bf)), BAD),
    (dict(qo=torch.zeros(1, 4, 64, dtype=bf).expand(4, 4, 64)), BAD),
    (dict(qo=torch.zeros(4, 4, 68, dtype=bf)[:, :, :64]), BAD), (dict(ko=torch.zeros(4, 4, 64, dtype=bf)), BAD),
    (dict(q=torch.zeros(4 * 4 * 64 + 4, dtype=bf)[4:].view(4, 4, 64)), BAD),
])
def test_refusals(lib, change, want):
    assert _call(lib, dict(_args(), **change)) == want
    assert binding.paged_attn_last_error_message()


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, float("inf")), (float("nan"), 1.0)])
def test_fp8_scales(lib, ks, vs):
    assert _call(lib, dict(_args(kv=torch.uint8), ks=ks, vs=vs)) == BAD


def test_head_dims(lib):
    for d, want in ((36, UNS), (520, UNS)):
        assert _call(lib, _args(D=d, R=4, axes=1)) == want


def test_binding_refuses_host_tensors_and_short_lists():
    a = _args()
    with pytest.raises(ValueError):
        binding.paged_attn_rope_cache_write(a["q"], a["k"], a["v"], a["pos"], a["tab"], a["sl"], a["kc"], a["vc"])
