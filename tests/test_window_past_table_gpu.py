"""A windowed sequence longer than its block-table row, so long that the window
starts past the row's last entry: no page of it can be read.  Its rows get out = 0
and lse = -inf (4-bit caches: the sink), the status word reports the length, and
the other sequences' rows are as with an empty one in its place (bf16, fp8 and 4-bit caches)."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _run(kind, lens, qsl, runs, window, sinks, fill):
    """Three sequences over tables of four pages; outputs filled beforehand."""
    g = torch.Generator(device="cuda").manual_seed(3)
    hq, hkv, d, nb = 8, 2, 64, 12
    i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    t = int(qsl[-1]) if qsl is not None else len(lens)
    q = torch.randn(t, hq, d, device="cuda", generator=g).to(torch.bfloat16)
    bt = torch.arange(nb, dtype=torch.int32, device="cuda").reshape(3, 4)
    out = torch.full_like(q, fill)
    lse = torch.full((t, hq), fill, device="cuda")
    opts = binding.make_options(sliding_window=window, sinks=sinks)
    meta = (bt, i32(lens), None if qsl is None else i32(qsl), runs)
    if kind == "q4":
        codes = [torch.randint(0, 256, (nb, 16, hkv, d // 2), device="cuda", dtype=torch.uint8, generator=g)
                 for _ in range(2)]
        scales = [torch.randint(0x30, 0x40, (nb, hkv, 16, d // 16), device="cuda", dtype=torch.uint8, generator=g)
                  for _ in range(2)]
        binding.paged_attn_decode_q4(q, *codes, *scales, *meta, out=out, lse=lse, options=opts)
    else:
        kv = [torch.randn(nb, 16, hkv, d, device="cuda", generator=g) for _ in range(2)]
        kv = [x.to(torch.bfloat16) if kind == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8) for x in kv]
        binding.paged_attn_decode(q, *kv, *meta, out=out, lse=lse, options=opts)
    torch.cuda.synchronize()
    return out, lse, binding.paged_attn_device_status(clear=True)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("qsl", [None, [0, 2, 5, 6]])
@pytest.mark.parametrize("long", [200, (1 << 31) - 1])
@pytest.mark.parametrize("sinks", [False, True])
def test_window_past_the_table_row(kind, qsl, long, sinks):
    runs = 1 if qsl is None else 3
    sk = torch.linspace(-1, 1, 8, device="cuda") if sinks else None
    # an empty sequence in its place: as many pages in the batch, so the same cut of them
    want = _run(kind, [64, 0, 40], qsl, runs, 32, sk, 7.0)
    rows = slice(1, 2) if qsl is None else slice(2, 5)
    for fill in (7.0, float("nan")):
        out, lse, status = _run(kind, [64, long, 40], qsl, runs, 32, sk, fill)
        assert status == binding.STATUS_SEQ_LEN
        assert (out[rows] == 0).all()
        if sinks and kind == "q4":
            assert torch.equal(lse[rows], sk.expand_as(lse[rows]))
        else:
            assert (lse[rows] == -np.inf).all()
        for a, b in ((out, want[0]), (lse, want[1])):
            for r in (slice(0, rows.start), slice(rows.stop, None)):
                assert torch.equal(a[r], b[r])
