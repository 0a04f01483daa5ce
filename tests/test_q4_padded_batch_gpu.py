"""4-bit decode of a padded batch (sequences of length 0, or without query tokens,
as a captured graph of a fixed batch has): its live sequences' pages are cut over
the CTAs as without the padding."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from test_parity_q4_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _padded(c, place, batch, no_tokens):
    """Case c's sequences at rows `place` of a batch; the others are empty, or have keys but no query tokens."""
    p = object.__new__(Case)
    p.__dict__.update(c.__dict__)
    p.lens = np.full(batch, 50 if no_tokens else 0, dtype=np.int32)
    p.lens[place] = c.lens
    p.bt = np.full((batch, max(4, c.bt.shape[1])), 0, dtype=np.int32)
    p.bt[place, :c.bt.shape[1]] = c.bt
    p.qlens = np.zeros(batch, dtype=np.int64)
    p.qlens[place] = c.qlens
    p.qsl = np.concatenate([[0], np.cumsum(p.qlens)]).astype(np.int32)
    return p


def _cut(c, grid):
    """Outputs, and every live unit's first CTA and number of pieces (the descriptors at the workspace's start)."""
    o = binding.make_options(num_ctas=grid)
    plan = binding.paged_attn_q4_plan(len(c.lens), c.hq, c.hkv, c.d, c.runs, options=o)
    ws = torch.zeros(plan["workspace_bytes"], dtype=torch.uint8, device="cuda")
    out, lse = c.run(num_ctas=grid, workspace=ws.data_ptr(), workspace_bytes=ws.numel())
    units = len(c.lens) * (c.hkv // plan["heads_per_cta"])
    d = ws[:16 * units].view(torch.int32).reshape(len(c.lens), -1, 4).cpu().numpy()[c.qlens > 0]
    return out, lse, d[..., 0], d[..., 1] & 0x3FFFFFFF


@pytest.mark.parametrize("no_tokens", [False, True])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
@pytest.mark.parametrize("lens,qlens,hq,hkv,d,batch,grid", [
    ([4096, 3000, 17, 1000], [1, 1, 1, 1], 8, 8, 128, 100, 300),
    ([900] * 8, [1] * 8, 8, 1, 64, 256, 150),
    ([2000, 500, 1], [3, 2, 1], 16, 2, 128, 64, 148),
    ([700, 90], [4, 1], 32, 4, 64, 33, 0)])
def test_padding_does_not_move_the_cut(lens, qlens, hq, hkv, d, batch, grid, where, no_tokens):
    c = Case(lens, qlens, hq=hq, hkv=hkv, d=d, seed=batch)
    n = len(lens)
    place = {"first": np.arange(n), "last": np.arange(batch - n, batch),
             "spread": np.sort(np.random.default_rng(batch).permutation(batch)[:n])}[where]
    want, got = _cut(c, grid), _cut(_padded(c, place, batch, no_tokens), grid)
    assert np.array_equal(want[2], got[2]) and np.array_equal(want[3], got[3])
    # (the batch's size chooses the merge's form, so sums may differ in their order)
    c.check(*want[:2])
    c.check(*got[:2])


def test_the_largest_batch_with_two_live_sequences():
    """8192 rows of which two have pages: the whole grid takes part."""
    c = Case([20000, 12000], [1, 1], hq=8, hkv=1, d=64, seed=5)
    p = _padded(c, [3000, 8191], 8192, False)
    out, lse, first, pieces = _cut(p, 148)
    busy = set()
    for f, n in zip(first.ravel(), pieces.ravel()):
        busy |= set(range(f, f + n))
    assert len(busy) >= 140
    c.check(out, lse)
