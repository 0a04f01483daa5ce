"""Sequences longer than their block-table rows, up to the largest length an int32 holds, in
decode over windows with first tokens and over shared prefixes: reported, nothing past the
row is read, and the other sequences' rows are right."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu
LONG = pytest.mark.parametrize("long", [5000, 2 ** 31 - 17, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1])


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield
    binding.paged_attn_device_status(clear=True)


def _others(b, run, who, long):
    """Outputs of the sequences but `who` are the oracle's when that one's length is `long`."""
    kept = b.lens.copy()
    out, lse = run()
    assert binding.paged_attn_device_status() == 0
    b.check(out, lse, *b.view)
    b.lens[who] = long
    got, gl = run()
    b.lens[:] = kept
    assert binding.paged_attn_device_status(clear=True) == binding.STATUS_SEQ_LEN
    rest = np.arange(len(kept)) != who
    wo, wl, spread = b.want(*b.view)
    # twice the output's rounding to bf16 and the weights' (2^-8 each, of the row's weighted |v|)
    assert (np.abs(got.double().cpu().numpy() - wo)[rest] <= (2.0 ** -7 * (np.abs(wo) + spread))[rest]).all()
    assert (np.abs(gl.double().cpu().numpy() - wl)[rest] <= 1e-4).all()


@LONG
@pytest.mark.parametrize("first", [0, 20])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_window(kv, first, long):
    b = Batch([64, 300, 90], hq=8, hkv=2, kv=kv)
    b.view = (70, first)

    def run():
        out, lse = b.buffers()
        binding.paged_attn_decode_window(*b.on_gpu(), 1, *b.view, b.scale, b.ks, b.vs, out=out, lse=lse,
                                         options=b.options())
        return out, lse
    _others(b, run, 1, long)


@LONG
@pytest.mark.parametrize("kw", [{}, {"disable_pdl": True}])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_shared_prefix(kv, kw, long):
    b = Batch([900 + i for i in range(40)], hq=16, hkv=4, kv=kv, groups=([0, 40], [890]))
    b.view = ()

    def run():
        out, lse = b.buffers()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        binding.paged_attn_decode_shared(*b.on_gpu(), 1, i32(b.groups[0]), i32(b.groups[1]), b.scale, b.ks, b.vs, out=out,
                                         lse=lse, options=b.options(**kw))
        return out, lse
    _others(b, run, 39, long)                                   # the longest: its row has no free entries
