"""paged_attn_decode_window against the float64 oracle."""
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


def _run(b, window, first, **kw):
    dev = b.on_gpu()
    out, lse = b.buffers()
    binding.paged_attn_decode_window(*dev, b.runs, window, first, b.scale, b.ks, b.vs, out=out, lse=lse,
                                     options=b.options(**kw))
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (16, 4), (17, 16), (50, 17), (100, 40), (3, 100), (1000, 5),
                                          (31, 0), (33, 33), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows(window, first, d, kv):
    b = Batch([1, 2, 15, 16, 17, 33, 64, 100, 300, 511], hq=8, hkv=2, d=d, kv=kv, seed=window)
    b.check(*_run(b, window, first), window, first)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,runs", [(1, 1, 1), (5, 5, 7), (16, 1, 4), (24, 3, 5), (64, 1, 1), (20, 10, 3), (28, 4, 2)])
def test_heads_and_runs(hq, hkv, runs, kv):
    lens = [runs, 20, 47, 129, 640, 1003]
    b = Batch(lens, [runs, 1, min(2, runs), runs, max(1, runs - 1), runs], hq=hq, hkv=hkv, kv=kv, sinks=runs > 2)
    b.check(*_run(b, 60, 20), 60, 20)


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("fp8", 128)])
def test_long_sequences_cut_into_many_pieces(kv, d):
    b = Batch([20011], hq=8, hkv=2, d=d, kv=kv)
    b.check(*_run(b, 15000, 100), 15000, 100)
    b = Batch([20011, 9000, 40], hq=4, hkv=4, d=d, kv=kv)
    b.check(*_run(b, 7001, 33), 7001, 33)


def test_per_token_scales():
    b = Batch([3, 90, 700, 1500], [1, 3, 2, 3], hq=8, hkv=2, kv="fp8", tokens=True)
    b.check(*_run(b, 200, 21), 200, 21)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("window,first,runs", [(20, 5, 1), (7, 20, 3), (40, 0, 2), (33, 31, 3)])
def test_hidden_slots_hold_nan(window, first, runs, kv):
    """Slots between the first tokens and the window, and past the end, are NaN, also in pages that are read."""
    lens = [50, 111, 300, 64, 16]
    b = Batch(lens, [runs] * 5, hq=8, hkv=2, kv=kv, tokens=kv == "fp8")
    want = b.want(window, first)
    nan = float("nan") if kv == "bf16" else 0x7F
    for i, L in enumerate(lens):
        end = -(-L // 16) * 16
        hidden = [j for j in range(end) if j >= L or first <= j < L - runs - window + 1]
        for j in hidden:
            page = b.bt[i, j // 16]
            b.k[page, j % 16], b.v[page, j % 16] = nan, nan
            if b.tk is not None:
                b.tk[page, :, j % 16] = b.tv[page, :, j % 16] = float("nan")
    free = sorted(set(range(b.k.shape[0])) - set(b.bt[b.bt >= 0].tolist()))
    b.k[free], b.v[free] = nan, nan
    out, lse = _run(b, window, first)
    clean = b.want(window, first)
    assert all(np.array_equal(x, y) for x, y in zip(want, clean))
    b.check(out, lse, window, first)


def test_nan_in_a_seen_key_is_not_lost():
    for cut in (0, 40):
        b = Batch([700, 700], hq=4, hkv=2, seed=3)
        b.k[b.bt[0, 43], 3, 0] = float("nan")
        out, lse = _run(b, 300, 4, num_ctas=cut)
        assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
        assert torch.isfinite(out[0, 2:]).all() and torch.isfinite(out[1]).all()
        b = Batch([700], hq=4, hkv=2, seed=3)
        b.q[0, 1] = float("nan")                          # every score of the head, in every piece
        out, lse = _run(b, 300, 4, num_ctas=cut)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]) and torch.isfinite(out[0, [0, 2, 3]]).all()


@pytest.mark.parametrize("sinks", [False, True])
def test_padded_batch_and_empty_rows(sinks):
    b = Batch([0, 2, 40, 0, 333, 50], [1, 4, 2, 0, 3, 0], hq=8, hkv=2, d=64, sinks=sinks, pad_rows=5)
    b.check(*_run(b, 21, 5), 21, 5, status=binding.STATUS_SEQ_LEN)


def test_padding_alone_sets_no_status():
    b = Batch([9, 0, 70], [2, 0, 1], hq=8, hkv=2, d=64, pad_rows=2)
    b.check(*_run(b, 16, 2), 16, 2)


def test_context_past_the_table_row_stays_in_bounds():
    b = Batch([64, 30], hq=4, hkv=2)
    b.lens[0] = 5000
    out, lse = _run(b, 40, 4)
    assert binding.paged_attn_device_status() & binding.STATUS_SEQ_LEN
    b.lens[0] = 64
    wo, _, _ = b.want(40, 4)
    assert np.abs(out[1].double().cpu().numpy() - wo[1]).max() < 1e-2


def test_bad_page_id_is_reported():
    b = Batch([64, 200], hq=4, hkv=2)
    b.bt[1, 0] = b.k.shape[0]
    _run(b, 40, 4)
    assert binding.paged_attn_device_status() & binding.STATUS_PAGE_RANGE
    b.bt[1, 5] = -7                                   # a page that nobody sees is not read
    b.bt[1, 0] = 0
    binding.paged_attn_device_status(clear=True)
    _run(b, 40, 4)
    assert binding.paged_attn_device_status() == 0


@pytest.mark.parametrize("kw", [dict(num_ctas=1), dict(num_ctas=7, min_pages_per_cta=1), dict(heads_per_cta=1),
                                dict(disable_pdl=True), dict(page_pairing=1), dict(page_pairing=2), dict(num_ctas=400)])
def test_launch_forms(kw):
    b = Batch([5, 700, 1000, 48], [2, 3, 1, 3], hq=8, hkv=2, kv="bf16")
    b.check(*_run(b, 333, 36, **kw), 333, 36)


def test_graphs_streams_and_prepared_calls():
    b = Batch([100, 1000, 3000], hq=8, hkv=2)
    dev = b.on_gpu()
    calls = [binding.prepare_decode_window(*dev, 1, w, 5, b.scale) for w in (100, 900)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls[0]()
    calls[1]()
    torch.cuda.synchronize()
    for c, w in zip(calls, (100, 900)):
        b.check(c.out, c.lse, w, 5)
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for c in calls:
        c.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, w in zip(calls, (100, 900)):
        b.check(c.out, c.lse, w, 5)


def test_strided_caches_and_outputs():
    b = Batch([100, 400], hq=8, hkv=2, d=64)
    dev = b.on_gpu()
    wide = torch.zeros(*b.k.shape[:2], 3, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :2, :64] = dev[1]
    dev[1] = wide[:, :, :2, :64]
    out = torch.full((2, 10, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 20), 7.0, device="cuda")
    binding.paged_attn_decode_window(*dev, 1, 50, 9, b.scale, out=out[:, :8, :64], lse=lse[:, :16:2])
    b.check(out[:, :8, :64], lse[:, :16:2], 50, 9)
    assert (out[:, 8:] == 7).all() and (out[..., 64:] == 7).all() and (lse[:, 1::2] == 7).all()
