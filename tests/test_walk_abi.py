"""Host checks of the decode calls over walks with a hole: what they refuse before
anything reaches the device (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import build as builder

BAD, UNS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED
bf, i32 = torch.bfloat16, torch.int32


@pytest.fixture(autouse=True)
def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.load()


def _args(T=3, Hq=8, Hkv=2, D=128, NB=10, B=3, MB=4, kv=bf, runs=1):
    return dict(q=torch.zeros(T, Hq, D, dtype=bf), k=torch.zeros(NB, 16, Hkv, D, dtype=kv),
                v=torch.zeros(NB, 16, Hkv, D, dtype=kv), bt=torch.zeros(B, MB, dtype=i32),
                sl=torch.ones(B, dtype=i32), qsl=None, out=torch.zeros(T, Hq, D, dtype=bf), lse=torch.zeros(T, Hq),
                runs=runs, window=8, first=2, scale=0.1, opts=None)


def _window(lib, a):
    r = [ctypes.byref(binding.tensor_desc(a[n])) for n in ("q", "k", "v", "bt", "sl", "qsl", "out", "lse")]
    return lib.paged_attn_decode_window(*r[:6], a["runs"], a["window"], a["first"], a["scale"], 1.0, 1.0, *r[6:],
                                        ctypes.byref(a["opts"]) if a["opts"] is not None else None, None)


def _shared(lib, a):
    gsl, lens = a.get("gsl", torch.tensor([0, 2], dtype=i32)), a.get("shared", torch.tensor([16], dtype=i32))
    r = [ctypes.byref(binding.tensor_desc(t)) for t in
         [a[n] for n in ("q", "k", "v", "bt", "sl", "qsl")] + [gsl, lens, a["out"], a["lse"]]]
    return lib.paged_attn_decode_shared(*r[:6], a["runs"], r[6], r[7], a["scale"], 1.0, 1.0, *r[8:],
                                        ctypes.byref(a["opts"]) if a["opts"] is not None else None, None)


CALLS = [_window, _shared]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("make", [
    lambda: _args(), lambda: _args(kv=torch.uint8), lambda: dict(_args(), lse=None), lambda: _args(D=64),
    lambda: dict(_args(T=7), qsl=torch.tensor([0, 2, 2, 4], dtype=i32), runs=2), lambda: _args(T=5),
    lambda: dict(_args(), opts=binding.make_options(num_ctas=5, heads_per_cta=2, disable_pdl=True)),
    lambda: _args(Hq=64, Hkv=1)])
def test_valid_calls_pass(lib, call, make):
    # every host check passed: without a GPU the call then fails at device set-up
    assert call(lib, make()) == binding.PA_ERR_CUDA, binding.paged_attn_last_error_message()


@pytest.mark.parametrize("call", CALLS)
def test_no_tokens_is_no_work(lib, call):
    assert call(lib, _args(T=0)) == binding.PA_OK


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,want", [
    (dict(q=torch.zeros(3, 8, 128)), BAD), (dict(out=torch.zeros(3, 8, 128)), BAD),
    (dict(out=torch.zeros(3, 4, 128, dtype=bf)), BAD), (dict(lse=torch.zeros(3, 4)), BAD),
    (dict(lse=torch.zeros(3, 8, dtype=bf)), BAD), (dict(k=torch.zeros(10, 16, 2, 128)), BAD),
    (dict(v=torch.zeros(10, 16, 2, 128, dtype=torch.uint8)), BAD), (dict(v=torch.zeros(9, 16, 2, 128, dtype=bf)), BAD),
    (dict(k=torch.zeros(10, 8, 2, 128, dtype=bf), v=torch.zeros(10, 8, 2, 128, dtype=bf)), UNS),
    (dict(k=torch.zeros(10, 16, 3, 128, dtype=bf), v=torch.zeros(10, 16, 3, 128, dtype=bf)), BAD),
    (dict(bt=torch.zeros(3, 4)), BAD), (dict(bt=torch.zeros(4, 3, dtype=i32).t()), BAD),
    (dict(bt=torch.zeros(3, 0, dtype=i32)), BAD), (dict(sl=torch.ones(2, dtype=i32)), BAD),
    (dict(sl=torch.ones(3, dtype=torch.int64)), BAD), (dict(runs=2), BAD), (dict(runs=0), BAD),
    (dict(qsl=torch.zeros(3, dtype=i32)), BAD), (dict(qsl=torch.zeros(8, dtype=i32)[::2]), BAD),
    (dict(q=torch.zeros(2, 8, 128, dtype=bf), out=torch.zeros(2, 8, 128, dtype=bf), lse=None), BAD),
    (dict(q=torch.zeros(3, 8, 256, dtype=bf)[..., :128]), BAD), (dict(scale=float("nan")), BAD),
    (dict(q=torch.zeros(3 * 8 * 128 + 4, dtype=bf)[4:].view(3, 8, 128)), BAD),
    (dict(out=torch.zeros(1, 8, 128, dtype=bf).expand(3, 8, 128)), BAD), (dict(lse=torch.zeros(1, 8).expand(3, 8)), BAD),
    (dict(opts=binding.make_options(sliding_window=5)), UNS), (dict(opts=binding.make_options(use_tcgen05=2)), UNS),
    (dict(opts=binding.make_options(num_ctas=1 << 20)), BAD), (dict(opts=binding.make_options(heads_per_cta=3)), BAD),
    (dict(opts=binding.make_options(segment_cost_pages=2)), UNS), (dict(opts=binding.make_options(wait_limit_us=-1)), BAD),
])
def test_refusals(lib, call, change, want):
    assert call(lib, dict(_args(), **change)) == want
    assert binding.paged_attn_last_error_message()


@pytest.mark.parametrize("call", CALLS)
def test_shapes_outside_the_envelope(lib, call):
    for a, want in ((_args(D=96), UNS), (_args(Hq=66, Hkv=1), UNS), (_args(Hq=9), BAD),
                    (dict(_args(Hq=32, T=9), qsl=torch.zeros(4, dtype=i32), runs=5), UNS)):
        assert call(lib, a) == want


def test_window_and_first_tokens(lib):
    for w, f in ((0, 1), (-3, 1), (4, -1)):
        assert _window(lib, dict(_args(), window=w, first=f)) == BAD


def test_window_token_scales(lib):
    z = lambda *s, **k: torch.zeros(*s, **k)
    good = z(10, 2, 16)
    ok = dict(k_token_scales=good, v_token_scales=good)
    assert _window(lib, dict(_args(kv=torch.uint8), opts=binding.make_options(**ok))) == binding.PA_ERR_CUDA
    assert _window(lib, dict(_args(), opts=binding.make_options(**ok))) == BAD
    for k in (z(9, 2, 16), z(10, 2, 16, dtype=bf), z(10, 16, 2).transpose(1, 2)):
        o = binding.make_options(k_token_scales=k, v_token_scales=good)
        assert _window(lib, dict(_args(kv=torch.uint8), opts=o)) == BAD
    o = binding.make_options(k_token_scales=good)
    assert _window(lib, dict(_args(kv=torch.uint8), opts=o)) == BAD


@pytest.mark.parametrize("gsl,shared,want", [
    (torch.tensor([0, 1, 3], dtype=i32), torch.tensor([16], dtype=i32), BAD),
    (torch.tensor([0, 1]), torch.tensor([16], dtype=i32), BAD), (torch.tensor([0, 1], dtype=i32), torch.tensor([16.0]), BAD),
    (torch.tensor([0, 9, 1], dtype=i32)[::2], torch.tensor([16], dtype=i32), BAD),
    (torch.tensor([0, 1, 2], dtype=i32), torch.tensor([16, 0, 16, 0], dtype=i32)[::2], BAD),
    (torch.zeros(5, dtype=i32), torch.zeros(4, dtype=i32), UNS), (None, torch.tensor([16], dtype=i32), BAD),
    (torch.tensor([0, 1], dtype=i32), None, BAD),
    (torch.tensor([0], dtype=i32), torch.zeros(0, dtype=i32), binding.PA_ERR_CUDA)])
def test_shared_lists(lib, gsl, shared, want):
    assert _shared(lib, dict(_args(), gsl=gsl, shared=shared)) == want


def test_shared_options(lib):
    z = torch.zeros(10, 2, 16)
    o = binding.make_options(k_token_scales=z, v_token_scales=z)
    assert _shared(lib, dict(_args(kv=torch.uint8), opts=o)) == UNS
    assert _shared(lib, dict(_args(), opts=binding.make_options(test_starve_cta=1))) == UNS


def test_shared_workspace_shapes(lib):
    for shape, want in (((4, 0, 8, 2, 128), UNS), ((1 << 27, 4, 8, 2, 128), UNS), ((-1, 4, 8, 2, 128), UNS),
                        ((4, 4, 9, 2, 128), BAD), ((4, 4, 8, 2, 128, binding.PA_BF16, 0), BAD),
                        ((4, 4, 8, 2, 128, binding.PA_BF16, 17), UNS)):
        with pytest.raises(binding.PagedAttnError) as e:
            binding.paged_attn_shared_workspace_size(*shape)
        assert e.value.status == want, shape
