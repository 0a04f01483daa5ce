"""paged_attn_decode_shared where the prefix kernel is sure to take part: launch forms
that share every prefix, and prefixes that are worth a part of their own.  The plan's list
of skipped pages (the workspace's first int32 a sequence) shows it."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu

FORMS = {"one after the other": {"disable_pdl": True}, "cut to 40": {"num_ctas": 40}, "side by side": {}}
form = pytest.mark.parametrize("form", list(FORMS))
short_form = pytest.mark.parametrize("form", list(FORMS)[:2])   # side by side, prefixes below 16 pages are not shared


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(b, form, dev=None, groups=None, skip=None):
    """(out, lse); the pages that each sequence left to its group must be `skip`, or some."""
    dev = dev or b.on_gpu()
    out, lse = b.buffers()
    gsl, shared = groups or b.groups
    n = binding.paged_attn_shared_workspace_size(
        b.q.shape[0], len(b.lens), b.hq, b.hkv, b.d, binding.PA_FP8_E4M3 if b.kv == "fp8" else binding.PA_BF16, b.runs,
        b.options(**FORMS[form]))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    binding.paged_attn_decode_shared(*dev, b.runs, _i32(gsl), _i32(shared), b.scale, b.ks, b.vs, out=out, lse=lse,
                                     options=b.options(workspace=ws.data_ptr(), workspace_bytes=n, **FORMS[form]))
    torch.cuda.synchronize()
    took = ws[:4 * len(b.lens)].view(torch.int32).cpu().numpy()
    assert (took == skip).all() if skip is not None else took.any(), took
    return out, lse


def _layouts(x):
    """The cache in rows of its heads, with room behind each head, and head by head."""
    nb, _, h, d = x.shape
    wide = torch.zeros(nb, 17, h + 1, d + 16, dtype=x.dtype, device="cuda")
    by_head = torch.zeros(nb, h, 16, d, dtype=x.dtype, device="cuda")
    yield x
    for y in (wide[:, :16, :h, :d], by_head.transpose(1, 2)):
        y.copy_(x)
        yield y


@form
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_every_layout_of_keys_beside_every_one_of_values(kv, d, form):
    # side by side: 40 x 68 pages x 3 heads x 59 ns at least, above the 304 us that are left to the sequences
    b = Batch([1100 + 9 * i for i in range(40)], hq=6, hkv=3, d=d, kv=kv, groups=([0, 40], [1090]))
    dev = b.on_gpu()
    first = None
    for k in _layouts(dev[1]):
        for v in _layouts(dev[2]):
            got = _run(b, form, [dev[0], k, v] + dev[3:], skip=1090 // 16)
            if first is None:
                first = got
                b.check(*got)
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@form
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_replays_over_new_lists(kv, form):
    """A captured call whose lists, lengths, tables and queries change between its replays: every kernel of it works
    on this replay's plan.  The word that says that the plan is there (behind the skipped pages) is taken back."""
    lens = np.concatenate([1200 + 5 * np.arange(60), [40] * 4])
    batches = [Batch(lens, hq=16, hkv=4, d=64, kv=kv, groups=g, seed=7)
               for g in (([0, 30, 60], [1190, 1000]), ([10, 50, 60], [1195, 160]), ([0, 60, 64], [700, 0]))]
    assert all((x.lens == lens).all() and x.bt.shape == batches[0].bt.shape for x in batches)
    pages = max(x.k.shape[0] for x in batches)
    dev = batches[0].on_gpu()
    for x in (1, 2):
        dev[x] = torch.zeros(pages, *dev[x].shape[1:], dtype=dev[x].dtype, device="cuda")
    lists = [_i32([0, 0, 0]), _i32([0, 0])]
    out, lse = batches[0].buffers()
    code = binding.PA_FP8_E4M3 if kv == "fp8" else binding.PA_BF16
    n = binding.paged_attn_shared_workspace_size(64, 64, 16, 4, 64, code, 1, batches[0].options(**FORMS[form]))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    call = binding.prepare_decode_shared(*dev, 1, *lists, batches[0].scale, batches[0].ks, batches[0].vs, out=out, lse=lse,
                                         options=batches[0].options(workspace=ws.data_ptr(), workspace_bytes=n, **FORMS[form]))
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    word = ws[256:264].view(torch.int64)
    for again in range(3):
        for b in batches:
            new = b.on_gpu() + [_i32(b.groups[0]), _i32(b.groups[1])]
            for x, y in zip(dev + lists, new):
                if y is not None:
                    x[:y.shape[0]].copy_(y)
            out.fill_(7.0)
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            assert int(word) == 0 and ws[:256].view(torch.int32).any()
            if again == 0:
                b.check(out, lse)
                b.got = out.clone(), lse.clone()
            assert torch.equal(out, b.got[0]) and torch.equal(lse, b.got[1])
