"""Decode calls in which warps give up on a wait while copies are on their way: the
consumers of one CTA do at once (test_give_up_cta), so the warps that wait for them wait
out the limit.  The call ends soon, within its buffers, and the next one is right."""
import time

import numpy as np
import pytest
import torch

import oracle
from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import workloads as wl
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield
    binding.paged_attn_device_status(clear=True)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _decode(b, dev, out, lse, **kw):
    binding.paged_attn_decode(*dev, b.runs, b.scale, b.ks, b.vs, out=out, lse=lse, options=b.options(**kw))


def _window(b, dev, out, lse, **kw):
    binding.paged_attn_decode_window(*dev, b.runs, 700, 20, b.scale, b.ks, b.vs, out=out, lse=lse, options=b.options(**kw))


def _shared(b, dev, out, lse, **kw):
    binding.paged_attn_decode_shared(*dev, b.runs, _i32(b.groups[0]), _i32(b.groups[1]), b.scale, b.ks, b.vs, out=out,
                                     lse=lse, options=b.options(**kw))


def _given_up(call, b, view, ctas=(1, 6), **kw):
    dev = b.on_gpu()
    for k in ctas:
        out, lse = b.buffers()
        t0 = time.perf_counter()
        call(b, dev, out, lse, wait_limit_us=1000, test_give_up_cta=k, **kw)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 2.0
        assert binding.paged_attn_device_status(clear=True) == binding.STATUS_TIMEOUT
        out, lse = b.buffers()
        call(b, dev, out, lse, **kw)
        b.check(out, lse, *view)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("call,view", [(_decode, ()), (_window, (700, 20))])
def test_split_kernel(call, view, kv):
    b = Batch(1000 + 37 * np.arange(24), 1 + np.arange(24) % 3, hq=8, hkv=4, kv=kv, seed=1)
    _given_up(call, b, view)


def test_token_scales():
    b = Batch(600 + 37 * np.arange(12), hq=8, hkv=4, kv="fp8", tokens=True, seed=3)
    _given_up(_window, b, (700, 20))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_sequences_behind_a_shared_prefix(kv):
    b = Batch(1400 + np.arange(40), hq=16, hkv=2, kv=kv, groups=([0, 40], [1390]), seed=2)
    _given_up(_shared, b, ())
    _given_up(_shared, b, (), num_ctas=20)


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_shared_prefix(kv, d):
    """Four CTAs of many steps each, pairs of tiles and single ones: the loaders, converters, product issuers
    and the other tile's softmax wait out the limit one after the other."""
    b = Batch(6000 + np.arange(40), hq=16, hkv=2, d=d, kv=kv, groups=([0, 40], [5990]), seed=6)
    _given_up(_shared, b, (), ctas=(1, 3), num_ctas=4)


@pytest.mark.parametrize("runs", [1, 5])
def test_tensor_memory_split_kernel(runs):
    b = Batch(1000 + 37 * np.arange(24), 1 + np.arange(24) % runs, hq=16, hkv=2, seed=4)
    _given_up(_decode, b, (), use_tcgen05=2)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_mla(kv):
    scale = 0.05 if kv == "fp8" else 1.0
    w = wl.make_mla_workload(wl.custom_mla_spec(num_q_heads=16, kv_dtype=kv, seq_lens=(700, 1000, 333, 901, 640, 1023),
                                                query_len_choices=(2,), kv_scale=scale, fp8_source_scale=scale, seed=5),
                             device="cuda")
    ref = oracle.run_mla_workload(w)
    for k in (1, 6):
        t0 = time.perf_counter()
        binding.mla_decode_workload(w, options=binding.make_options(use_tcgen05=1, wait_limit_us=1000, test_give_up_cta=k))
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 2.0
        assert binding.paged_attn_device_status(clear=True) & binding.STATUS_TIMEOUT
        out, lse = binding.mla_decode_workload(w, options=binding.make_options(use_tcgen05=1))
        assert binding.paged_attn_device_status() == 0
        # the bounds of the parity tests of these kernels
        assert np.abs(out.float().cpu().numpy() - ref[0]).max() <= (2e-2 if kv == "fp8" else 1e-2)
        assert np.abs(lse.cpu().numpy() - ref[1]).max() <= 1e-3
