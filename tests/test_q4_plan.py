"""What paged_attn_q4_plan reports: the layout of its struct, and the launch forms
that the sequences' metadata leaves room for (warps a head, CTAs an SM)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding


def test_plan_struct_keeps_its_layout():
    """warps_per_head lies in what was padding: the other fields and the size are as before it."""
    f = binding.PaPlan
    assert ctypes.sizeof(f) == 56 and f.warps_per_head.offset == 36 and f.workspace_bytes.offset == 40
    assert f.page_pairing.offset == 32 and f.variant.offset == 48 and f.block_pages.offset == 52


@pytest.mark.gpu
def test_plan_reports_two_pages_a_step(cuda_lib):
    p = binding.paged_attn_q4_plan(3, 32, 8, 128)
    assert p["variant"] == 4 and p["page_pairing"] == 1 and p["block_pages"] == 2 and p["warps_per_head"] == 1
    assert binding.paged_attn_plan(3, 32, 8, 128)["warps_per_head"] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,hkv,d,rows,warps,per_sm", [
    (3000, 8, 8, 64, 1, 1, 1),        # the metadata leaves room for one CTA an SM
    (100, 8, 8, 64, 1, 1, 2), (100, 8, 4, 128, 1, 2, 2), (100, 8, 1, 128, 1, 8, 1),
    (8192, 16, 1, 128, 1, 4, 1),      # ... for four warps a head, not eight
    (8192, 32, 2, 128, 1, 2, 1)])     # ... for two, not four
def test_launch_forms_and_their_results(cuda_lib, b, hq, hkv, d, rows, warps, per_sm):
    from test_parity_q4_gpu import Case
    p = binding.paged_attn_q4_plan(b, hq, hkv, d, rows)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert p["warps_per_head"] == warps and p["num_ctas"] == per_sm * sms
    r = np.random.default_rng(b)
    lens = np.where(r.random(b) < 0.2, r.integers(1, 40, b), 0)
    lens[[7, 50]] = 900, 130
    c = Case(lens, (lens > 0).astype(np.int64), hq=hq, hkv=hkv, d=d, seed=rows)
    binding.paged_attn_device_status(clear=True)
    c.check(*c.run())
