"""paged_attn_decode_q4 against the float64 oracle, every output element within the
bound that its own row's weights and values give (oracle.cache_q4.decode_with_bounds):
long contexts, whose outputs are far below the values, and sinks above the scores."""
import numpy as np
import pytest
import torch

from oracle import cache_q4
from paged_kv_decode_06_gb300 import binding
from test_oracle_q4_bounds import bounds, needle_case
from test_parity_q4_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def inside(out, lse, want):
    wo, wl, to, tl = want
    go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    live = ~np.isnan(wl)
    inf = np.isinf(wl)
    assert np.array_equal(gl[inf], wl[inf]) and np.isfinite(gl[live]).sum() == (live & ~inf).sum()
    ok = live & ~inf
    assert (np.abs(go - wo)[live] <= to[live]).all(), np.nanmax((np.abs(go - wo) / to)[live])
    assert (np.abs(gl[ok] - wl[ok]) <= tl[ok]).all(), np.max((np.abs(gl - wl) / tl)[ok])


def check(c, status=0, **kw):
    """A Case of the parity tests, within the bounds of its rows."""
    out, lse = c.run(**kw)
    assert binding.paged_attn_device_status(clear=True) == status
    want = cache_q4.decode_with_bounds(c.q.double().numpy(), c.codes, c.scales, c.bt, c.lens, c.qsl, c.scale, c.k_scale,
                                       c.v_scale, c.window, c.sinks)
    inside(out, lse, want)
    return want


def check_needles(c, **kw):
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    q = torch.from_numpy(c["q"].astype(np.float32)).to(torch.bfloat16).cuda()
    sinks = None if c["sinks"] is None else dev(c["sinks"])
    out, lse = binding.paged_attn_decode_q4(
        q, *map(dev, (*c["codes"], *c["scales"], c["bt"], c["lens"])), None, 1, c["scale"], 0.02, 0.03,
        options=binding.make_options(sliding_window=c["window"], sinks=sinks, **kw))
    inside(out, lse, bounds(c))


@pytest.mark.parametrize("ctas", [0, 1, 7])
@pytest.mark.parametrize("L,d,hq,hkv,window", [(20000, 64, 64, 1, 0), (20000, 64, 8, 8, 0), (9000, 128, 32, 4, 0),
                                               (5000, 128, 16, 1, 700), (33, 64, 8, 2, 0)])
def test_rows_that_look_at_one_token(L, d, hq, hkv, window, ctas):
    check_needles(needle_case(L, d, hq, hkv, seed=L + hq, window=window), num_ctas=ctas)


@pytest.mark.parametrize("lens,qlens,hq,hkv,d,window", [
    ([20000], None, 8, 1, 64, 0), ([6000, 300, 1], None, 8, 2, 128, 0), ([3000, 2000], [4, 2], 16, 2, 128, 0),
    ([3000, 900], [3, 4], 8, 2, 64, 1024), ([700] * 40, None, 8, 1, 64, 0)])
@pytest.mark.parametrize("gain", [0.05, 1.0])
def test_long_contexts(lens, qlens, hq, hkv, d, window, gain):
    """Weights alike (gain 0.05) and uneven ones."""
    check(Case(lens, qlens, hq=hq, hkv=hkv, d=d, window=window, seed=len(lens) + d, q_gain=gain))


@pytest.mark.parametrize("above", [5.0, 10.0, 14.0, 18.0, 25.0, 60.0])
@pytest.mark.parametrize("lens,qlens,hq,hkv,d,ctas", [
    ([512], None, 8, 8, 128, 0), ([600, 40], None, 8, 1, 64, 0), ([600, 40], [3, 2], 16, 2, 128, 5),
    ([1500, 300], [4, 4], 32, 4, 64, 0)])
def test_sinks_above_the_scores(above, lens, qlens, hq, hkv, d, ctas):
    """Sinks up to 60 nats above the largest score: the keys' weights keep their relative precision, whatever
    piece or warp the sink is counted in."""
    c = Case(lens, qlens, hq=hq, hkv=hkv, d=d, seed=int(above), q_gain=0.2)
    top = 0.0
    for h in range(hq):
        k = cache_q4.dequantise_rows(c.codes[0], c.scales[0].transpose(0, 2, 1, 3), c.k_scale)[:, :, h // (hq // hkv)]
        top = max(top, c.scale * np.abs(k @ c.q[:, h].double().numpy().T).max())
    c.sinks = (top + above + np.linspace(0, 1, hq)).astype(np.float32)
    check(c, num_ctas=ctas)


@pytest.mark.parametrize("lens,qlens,hq,hkv,d,window,ctas", [
    ([60, 17], None, 8, 8, 128, 0, 1),                 # finished in one warp
    ([60, 17], None, 8, 8, 128, 0, 0),
    ([400, 90], None, 8, 1, 64, 0, 1),                 # ... by eight warps
    ([900, 300], [2, 3], 16, 2, 128, 0, 9),            # cut
    ([900, 70], None, 32, 8, 64, 0, 300),
    ([2, 0, 40], [4, 2, 1], 8, 2, 128, 0, 3),          # rows without keys, an empty context
    ([200, 100], [8, 3], 8, 2, 64, 3, 20)])            # rows whose window starts in a later piece
def test_sinks_without_a_finite_value(lens, qlens, hq, hkv, d, window, ctas):
    """A NaN sink makes its head's rows NaN, +inf takes all weight, -inf is no sink."""
    c = Case(lens, qlens, hq=hq, hkv=hkv, d=d, window=window, seed=hq + ctas)
    plain = cache_q4.decode_with_bounds(c.q.double().numpy(), c.codes, c.scales, c.bt, c.lens, c.qsl, c.scale,
                                        c.k_scale, c.v_scale, window, None)
    c.sinks = np.tile(np.array([np.nan, np.inf, -np.inf, -np.inf], dtype=np.float32), hq // 4)
    out, lse = c.run(num_ctas=ctas, min_pages_per_cta=1)
    assert torch.isnan(out[:, 0::4]).all() and torch.isnan(lse[:, 0::4]).all()
    assert (out[:, 1::4] == 0).all() and (lse[:, 1::4] == np.inf).all()
    for h in (2, 3):
        inside(out[:, h::4], lse[:, h::4], [x[:, h::4] for x in plain])


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 60, (1 << 31) - 2000, 1 << 30])
def test_windows_of_any_size(window):
    """A window wider than any context is none, also for runs longer than their contexts."""
    check(Case([1, 30, 700], [8, 33, 3], hq=8, hkv=8, d=64, window=window, seed=4), status=binding.STATUS_SEQ_LEN)
