"""NaN and infinities through paged_attn_rope_cache_write, at slots that are written: they
stay in their own pair, a bf16 cache keeps them, an fp8 cache has NaN's code and the largest
codes (448) for infinities."""
import numpy as np
import pytest
import torch

from oracle import rope
from oracle.cache_write import e4m3fn_encode
from paged_kv_decode_06_gb300 import binding
from tests.test_rope_gpu import Case, _bits

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _codes(rows, scale):
    """Codes of float32 rows; NaN's and infinities' by their rule."""
    x = (rows / np.float32(scale)).astype(np.float64)
    fine = np.isfinite(x)
    codes = e4m3fn_encode(np.where(fine, x, 0.0)).astype(np.uint8)
    codes[np.isnan(x)] = 0x7F
    codes[x == np.inf], codes[x == -np.inf] = 0x7E, 0xFE
    return codes


def _same(got, want, is_nan):
    """Bits equal, NaN of any sign and payload beside NaN."""
    return (is_nan(got) == is_nan(want)).all() and (got == want)[~is_nan(want)].all()


NAN_OF = {"bf16": lambda b: (b & 0x7FFF) > 0x7F80, "fp8": lambda c: (c & 0x7F) == 0x7F}


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,d,rot", [(8, 64, 64), (9, 96, 32), (7, 48, 12), (6000, 64, 32), (6000, 48, 20)])
def test_special_values_stay_in_their_pair(t, d, rot, neighbours, kv):
    c = Case(t, 6, 3, d, rot, 3, kv, neighbours)
    c.slots[:] = np.random.default_rng(1).permutation(c.nb * 16)[:t]            # every token is written
    c.pos[:] = np.random.default_rng(2).integers(1, 300, c.pos.shape)           # no sine is zero
    last = d - 1
    for x, h in ((c.q, 5), (c.k, 2), (c.v, 1)):
        x[0, h, 0], x[1, h, 1], x[2, h, last] = NAN, INF, -INF
        x[3, 0, rot // 2], x[4, h, rot // 2 - 1] = -INF, NAN
        x[5, h, 0], x[5, h, 1 if neighbours else rot // 2] = INF, INF           # both of a pair
    qo, ko = c.run(key_out=True)
    assert binding.paged_attn_device_status() == 0
    rot_rows = lambda x: rope.rotate(x.float().cpu().numpy(), c.pos, c.table, c.axis, neighbours, np.float32)
    with np.errstate(invalid="ignore"):
        q, k, v = rot_rows(c.q), rot_rows(c.k), c.v.float().cpu().numpy()
    bf = lambda x: np.where(np.isnan(x), np.uint16(0x7FC0), rope.bf16_bits(np.where(np.isnan(x), 0, x)))
    assert _same(_bits(qo), bf(q), NAN_OF["bf16"]) and _same(_bits(ko), bf(k), NAN_OF["bf16"])
    page, slot = c.slots // 16, c.slots % 16
    for cache, rows, scale in ((c.kc, k, c.ks), (c.vc, v, c.vs)):
        with np.errstate(invalid="ignore", over="ignore"):
            want = bf(rows) if kv == "bf16" else _codes(rows, scale)
        assert _same(_bits(cache)[page, slot], want, NAN_OF[kv])
        hit = NAN_OF[kv](want) | (((want & 0x7FFF) == 0x7F80) if kv == "bf16" else ~np.isfinite(rows))
        assert 0 < int(hit.sum()) <= 2 * 7                                      # their own pairs and nothing else
