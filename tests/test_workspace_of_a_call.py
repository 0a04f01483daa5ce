"""The workspace that a decode call takes where its options have none: its size is kept
by everything it depends on (no GPU: a plan that stands in for the library's).
The descriptors of token scales live as long as the options that point to them."""
import gc
import weakref

import pytest
import torch

from paged_kv_decode_06_gb300 import binding

CPU = torch.device("cpu")


def _plan(*shape, options=None):
    o = options
    scales = 0 if o is None else bool(o.k_token_scales) + bool(o.v_token_scales)
    rest = (0,) * 5 if o is None else (o.num_ctas, o.min_pages_per_cta, o.heads_per_cta, o.page_pairing, o.use_tcgen05)
    return {"workspace_bytes": 256 * (1 + 5 * scales + sum((k + 2) * v for k, v in enumerate(rest)) + sum(shape))}


def _bytes(options):
    return binding._with_workspace(options, (1, 2, 3), CPU, _plan)[0].workspace_bytes


@pytest.fixture(autouse=True)
def _fresh():
    binding._WORKSPACE_BYTES.clear()
    yield
    binding._WORKSPACE_BYTES.clear()


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("kw", [dict(k_token_scales=torch.zeros(1, 2, 16), v_token_scales=torch.zeros(1, 2, 16)),
                                dict(num_ctas=3), dict(min_pages_per_cta=3), dict(heads_per_cta=2), dict(page_pairing=2),
                                dict(use_tcgen05=2)])
def test_a_size_is_kept_for_its_own_options(kw, first):
    calls = [None, binding.make_options(**kw)]
    for o in calls[::-1] if first else calls:
        assert _bytes(o) == _plan(1, 2, 3, options=o)["workspace_bytes"]


def test_the_token_scales_descriptors_live_as_long_as_a_calls_options():
    scales = torch.zeros(1, 2, 16)
    o = binding.make_options(k_token_scales=scales, v_token_scales=scales)
    kept = [weakref.ref(d) for d in o._tok_descs]
    mine, ws = binding._with_workspace(o, (1, 2, 3), CPU, _plan)
    del o
    binding._DESC_CACHE.clear()                      # (another place that may keep them for a while)
    gc.collect()
    assert all(d() is not None for d in kept)
    assert mine.k_token_scales.contents.data == scales.data_ptr()
