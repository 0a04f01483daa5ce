"""The binding's side of the 4-bit and page calls: missing tensors, and caches held in
torch's packed float4 type."""
import pytest
import torch

from paged_kv_decode_06_gb300 import binding

float4 = getattr(torch, "float4_e2m1fn_x2", None)
needs_float4 = pytest.mark.skipif(float4 is None, reason="this torch has no packed float4 type")


@pytest.mark.parametrize("call", [
    lambda: binding.paged_attn_cache_write_q4(*[None] * 7),
    lambda: binding.paged_attn_pages_copy([], None, None),
    lambda: binding.paged_attn_pages_fork([], *[None] * 6)])
def test_missing_tensors_are_invalid_arguments(monkeypatch, call):
    monkeypatch.setattr(binding, "load", lambda: None)          # refused before the library is called
    with pytest.raises(binding.PagedAttnError) as e:
        call()
    assert e.value.status == binding.PA_ERR_INVALID_ARG


@needs_float4
def test_float4_is_the_packed_code_type():
    codes = torch.zeros(3, 16, 2, 32, dtype=torch.uint8).view(float4)
    d = binding.tensor_desc(codes, binding._fp4_code)
    assert d.dtype == binding.PA_FP4_E2M1X2 and list(d.shape) == [3, 16, 2, 32] and list(d.stride)[:2] == [1024, 64]
    assert binding.tensor_desc(codes, binding._bytes_code).dtype == binding.PA_FP8_E4M3     # a byte, for page moves


@pytest.mark.gpu
@needs_float4
def test_float4_caches_are_written_read_decoded_and_copied(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    key, val, q, slots = rows(40, 2, 64), rows(40, 2, 64), rows(1, 8, 64), torch.arange(40, device="cuda").int()
    got = []
    for packed in (False, True):
        codes = [torch.zeros(6, 16, 2, 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(6, 2, 16, 4, dtype=torch.uint8, device="cuda") for _ in range(2)]
        c = [x.view(float4) for x in codes] if packed else codes
        s = [x.view(torch.float8_e4m3fn) for x in scales] if packed else scales
        binding.paged_attn_cache_write_q4(key, val, slots, *c, *s, 0.02, 0.02)
        binding.paged_attn_pages_copy([*c, *s], i32(0, 1, 2), i32(3, 4, 5))
        back = binding.paged_attn_cache_read_q4(slots, *c, *s, k_scale=0.02, v_scale=0.02)
        out = binding.paged_attn_decode_q4(q, *c, *s, i32(3, 4, 5)[None], i32(40), k_scale=0.02, v_scale=0.02)
        call = binding.prepare_decode_q4(q, *c, *s, i32(3, 4, 5)[None], i32(40), k_scale=0.02, v_scale=0.02)
        got.append([*codes, *scales, *back, *out, *call()])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][0].any() and (got[0][4] != 0).any()
    assert binding.paged_attn_device_status() == 0
