"""Decode calls whose waits are allowed a microsecond: some of them give up while copies
are on their way.  The call ends soon, within its buffers, and the next one is right."""
import time

import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
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


def _hurried(call, b, view, **kw):
    """Calls with a limit of 1 us over caches that no L2 line holds, then an ordinary one."""
    dev = b.on_gpu()
    big = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    out, lse = b.buffers()
    t0 = time.perf_counter()
    for _ in range(5):
        big.zero_()
        call(b, dev, out, lse, wait_limit_us=1, **kw)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert binding.paged_attn_device_status(clear=True) in (0, binding.STATUS_TIMEOUT)
    out, lse = b.buffers()
    call(b, dev, out, lse, **kw)
    b.check(out, lse, *view)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("call,view", [(_decode, ()), (_window, (700, 20))])
def test_split_kernel(call, view, kv):
    b = Batch(1000 + 37 * np.arange(24), 1 + np.arange(24) % 3, hq=8, hkv=4, kv=kv, seed=1)
    _hurried(call, b, view)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_shared_prefix(kv):
    b = Batch(1400 + np.arange(40), hq=16, hkv=2, kv=kv, groups=([0, 40], [1390]), seed=2)
    _hurried(_shared, b, ())
    _hurried(_shared, b, (), num_ctas=20)


def test_token_scales():
    b = Batch(600 + 37 * np.arange(12), hq=8, hkv=4, kv="fp8", tokens=True, seed=3)
    _hurried(_window, b, (700, 20))
