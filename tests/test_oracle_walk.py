"""Pins of the oracle of walks with a hole (no GPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import walk
from tests.walk_cases import Batch


def _bits(x):
    return x.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("window", [0, 5, 40])
@pytest.mark.parametrize("sinks", [False, True])
def test_without_first_tokens_it_is_the_window_oracle(window, sinks):
    b = Batch([1, 17, 64, 9], [1, 3, 2, 4], hq=6, hkv=3, d=64, sinks=sinks)
    out, lse, _ = b.want(window)
    ro, rl = oracle.paged_decode_attention(_bits(b.q), _bits(b.k), _bits(b.v), b.bt, b.lens, b.qsl, b.scale,
                                           sliding_window=window, sinks=b.sinks)
    assert np.allclose(out, ro, atol=1e-12) and np.allclose(lse, rl, atol=1e-12)


def test_visible_is_the_union():
    assert np.flatnonzero(walk.visible(9, 12, 3, 2)).tolist() == [0, 1, 7, 8, 9]
    assert np.flatnonzero(walk.visible(1, 12, 3, 5)).tolist() == [0, 1]
    assert np.flatnonzero(walk.visible(5, 12, 0, 0)).tolist() == [0, 1, 2, 3, 4, 5]
    assert not walk.visible(-1, 4, 3, 2).any()


def test_first_tokens_against_a_list_of_keys():
    b = Batch([50], hq=2, hkv=1, d=64)
    k, v = b.values()
    out, lse, spread = b.want(7, 3)
    rows = [0, 1, 2] + list(range(43, 50))
    kk = np.stack([k[b.bt[0, j // 16], j % 16, 0] for j in rows])
    vv = np.stack([v[b.bt[0, j // 16], j % 16, 0] for j in rows])
    s = np.float64(np.float32(b.scale)) * b.q.double().numpy()[0] @ kk.T
    p = np.exp(s) / np.exp(s).sum(-1, keepdims=True)
    assert np.allclose(out[0], p @ vv) and np.allclose(lse[0], np.log(np.exp(s).sum(-1)))
    assert (spread >= np.abs(out)).all()


def test_hidden_slots_may_hold_anything():
    b = Batch([40, 33], hq=2, hkv=1, d=64)
    a = b.want(5, 3)
    for i, L in enumerate((40, 33)):
        for j in range(3, L - 5):
            b.k[b.bt[i, j // 16], j % 16] = float("nan")
            b.v[b.bt[i, j // 16], j % 16] = float("inf")
    c = b.want(5, 3)
    assert all(np.array_equal(x, y) for x, y in zip(a, c))


def test_empty_rows():
    b = Batch([0, 2, 5], [1, 4, 0], hq=2, hkv=1, d=64, sinks=True)
    out, lse, _ = b.want(4, 1)
    assert (out[:3] == 0).all() and (lse[:3] == b.sinks.astype(np.float64)).all() and np.isfinite(lse).all()
    b.sinks = None
    out, lse, _ = b.want(4, 1)
    assert (out[:3] == 0).all() and np.isneginf(lse[:3]).all() and np.isfinite(lse[3:]).all()


def test_shared_pages_are_the_same_pages():
    b = Batch([70, 66, 90], groups=([0, 2, 3], [64, 40]))
    assert (b.bt[0, :4] == b.bt[1, :4]).all() and len(set(b.bt[b.bt >= 0].tolist())) == 5 + 1 + 6
