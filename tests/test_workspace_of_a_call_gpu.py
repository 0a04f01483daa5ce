"""A shape whose launch plan differs with per-token scales: calls with and without them, in
either order, each have the workspace they need."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", [(True, False), (False, True)])
def test_windows_with_and_without_token_scales(cuda_lib, order):
    lens = 1 + np.arange(5400) % 7
    binding._WORKSPACE_BYTES.clear()
    binding.paged_attn_device_status(clear=True)
    sizes = {}
    for tokens in order:
        b = Batch(lens, hq=128, hkv=8, d=128, kv="fp8", tokens=tokens, seed=1)
        dev = b.on_gpu()
        sizes[tokens] = binding.paged_attn_plan(5400, 128, 8, 128, binding.PA_FP8_E4M3, 1, b.options())["workspace_bytes"]
        call = lambda o: binding.paged_attn_decode_window(*dev, 1, 5, 1, b.scale, b.ks, b.vs, options=o)
        out, lse = call(b.options())
        ws = torch.empty(sizes[tokens], dtype=torch.uint8, device="cuda")
        want = call(b.options(workspace=ws.data_ptr(), workspace_bytes=sizes[tokens]))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.isfinite(lse).all()
        assert binding.paged_attn_device_status() == 0
    assert sizes[False] > sizes[True]
