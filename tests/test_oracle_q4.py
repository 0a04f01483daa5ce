"""Pins of the 4-bit cache's and the page operations' oracles (CPU)."""
import numpy as np
import pytest
import torch

from oracle import cache_q4, pages


def _bits(x):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_e2m1_grid_and_ties():
    codes = np.arange(16, dtype=np.uint8)
    v = cache_q4.e2m1_to_float64(codes)
    # sign, exponent (bias 1), mantissa written out
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        want = (-1) ** s * (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))
        assert v[c] == want
    assert np.array_equal(cache_q4.e2m1_encode(v), codes)
    # midpoints go to the neighbour with the even code
    mid = (v[:7] + v[1:8]) / 2
    assert cache_q4.e2m1_encode(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert cache_q4.e2m1_encode(-mid).tolist() == [8, 10, 10, 12, 12, 14, 14]
    assert cache_q4.e2m1_encode(np.array([5.1, 1e9, np.inf])).tolist() == [7, 7, 7]


@pytest.mark.parametrize("scale", [1.0, 0.05, 3.7e-3])
def test_rows_read_back_within_half_a_step(scale):
    """An e2m1 step is at most 2 (between 4 and 6), and S is within 2^-4 of amax / (6 s), so a
    value is off by at most half a step, amax / 6 * (1 + 2^-4), or by a clipping of amax / 16, which
    is less.  Where S saturates (amax > 448 * 6 s) the clipping is amax - 2688 s."""
    r = np.random.default_rng(0)
    x = r.standard_normal((40, 3, 64)) * np.exp(r.standard_normal((40, 3, 1)))
    bits = _bits(x)
    c, s = cache_q4.quantise_rows(bits, scale)
    assert c.shape == (40, 3, 32) and s.shape == (40, 3, 4)
    back = cache_q4.dequantise_rows(c, s, scale)
    xb = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double().numpy()
    amax = np.abs(xb.reshape(40, 3, 4, 16)).max(-1, keepdims=True)
    err = np.abs(back - xb).reshape(40, 3, 4, 16)
    clip = np.maximum(0.0, amax - 448 * 6 * float(np.float32(scale)))
    assert (err <= amax / 6 * (1 + 2.0 ** -4) + clip + 1e-12).all()


def test_zero_nan_and_infinite_groups():
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[0, 0, 1] = -0.0
    x[0, 0, 16:32] = 1.0
    x[0, 0, 20] = np.nan
    x[0, 0, 32:48] = 1.0
    x[0, 0, 40] = -np.inf
    x[0, 0, 48:64] = -6.0
    c, s = cache_q4.quantise_rows(_bits(x), 1.0)
    back = cache_q4.dequantise_rows(c, s, 1.0)[0, 0]
    assert s[0, 0].tolist() == [0, 0x7F, 0x7E, 0x38]
    assert (c[0, 0, :16] == 0).all()
    assert (back[:16] == 0).all() and np.isnan(back[16:32]).all()
    assert back[40] == -6 * 448 and (back[48:] == -6).all()


def test_rows_land_at_their_slots():
    r = np.random.default_rng(1)
    x = _bits(r.standard_normal((5, 2, 32)))
    codes = r.integers(0, 256, (3, 16, 2, 16)).astype(np.uint8)
    scales = r.integers(0, 127, (3, 2, 16, 2)).astype(np.uint8)
    slots = [17, -1, 0, 48, 47]                     # 48 is past the pool
    c, s = cache_q4.write_rows(x, slots, codes, scales, 0.5)
    qc, qs = cache_q4.quantise_rows(x, 0.5)
    assert np.array_equal(c[1, 1], qc[0]) and np.array_equal(s[1, :, 1], qs[0])
    assert np.array_equal(c[2, 15], qc[4]) and np.array_equal(c[0, 0], qc[2])
    changed = (c != codes).any(axis=(2, 3))
    assert changed.sum() <= 3
    back = cache_q4.read_rows(slots, c, s, 0.5, np.full((5, 2, 32), 9.0))
    assert (back[1] == 9).all() and (back[3] == 9).all()
    assert np.array_equal(back[0], cache_q4.dequantise_rows(qc[0], qs[0], 0.5))


def test_decode_oracle_against_dense_attention():
    r = np.random.default_rng(2)
    codes = [r.integers(0, 256, (9, 16, 2, 32)).astype(np.uint8) for _ in range(2)]
    scales = [r.integers(1, 0x60, (9, 2, 16, 4)).astype(np.uint8) for _ in range(2)]
    bt = r.permutation(9).reshape(3, 3)
    lens, qsl = np.array([1, 40, 0]), np.array([0, 1, 4, 5])
    q = r.standard_normal((6, 4, 64))
    sinks = r.standard_normal(4)
    out, lse = cache_q4.decode(q, codes, scales, bt, lens, qsl, 0.01, 1.0, 1.0, window=20, sinks=sinks)
    k, v = [torch.from_numpy(cache_q4.dequantise_rows(codes[x][bt[1]].reshape(48, 2, 32),
                                                      scales[x][bt[1]].transpose(0, 2, 1, 3).reshape(48, 2, 4), 1.0))
            for x in range(2)]
    for t in range(3):
        pos = 37 + t
        for h in range(4):
            s = 0.01 * (k[pos - 19:pos + 1, h // 2] @ torch.from_numpy(q[1 + t, h]))
            w = torch.softmax(torch.cat([s, torch.tensor([sinks[h]])]), 0)
            assert np.allclose(out[1 + t, h], (w[:-1] @ v[pos - 19:pos + 1, h // 2]).numpy(), rtol=1e-12)
            assert np.isclose(lse[1 + t, h], np.logaddexp(torch.logsumexp(s, 0).item(), sinks[h]), rtol=1e-12)
    assert (out[4] == 0).all() and np.allclose(lse[4], sinks) and np.isnan(out[5]).all()


def _pool(r, nb, rows, cols, lens):
    order = r.permutation(nb)
    bt, ref, at = np.full((rows, cols), -1, dtype=np.int32), np.zeros(nb, dtype=np.int32), 0
    for i, n in enumerate(lens):
        k = -(-n // 16)
        bt[i, :k] = order[at:at + k]
        ref[order[at:at + k]] = 1
        at += k
    return bt, np.array(lens, dtype=np.int32), ref, order[at:]


def test_fork_then_free_restores_the_pool():
    r = np.random.default_rng(3)
    bt, sl, ref, spare = _pool(r, 30, 6, 4, [33, 16, 60, 0, 0, 0])
    cache = r.integers(0, 99, (30, 7))
    new = np.array([spare[0], spare[1], spare[2]], dtype=np.int32)
    before = (bt[:3].copy(), sl.copy(), ref.copy())
    assert pages.fork([cache], bt, sl, ref, [0, 1, 0], [3, 4, 5], new) == 0
    assert sl.tolist() == [33, 16, 60, 33, 16, 33] and new.tolist() == [spare[0], -1, spare[2]]
    assert ref[bt[0, 0]] == 3 and ref[bt[0, 2]] == 1 and (cache[spare[0]] == cache[bt[0, 2]]).all()
    assert bt[3].tolist()[:3] == [bt[0, 0], bt[0, 1], spare[0]]
    st, ids, n = pages.free(bt, sl, ref, [3, 4, 5, 4])
    assert st == 0 and n == (before[2] == 0).sum() and (np.diff(ids[:n]) > 0).all()
    assert np.array_equal(ref, before[2]) and np.array_equal(sl, before[1])


def test_refused_forks_change_nothing():
    r = np.random.default_rng(4)
    bt, sl, ref, spare = _pool(r, 20, 5, 3, [33, 20, 0, 0, 0])
    state = [x.copy() for x in (bt, sl, ref)]
    new = np.array([spare[0], spare[0], spare[1], bt[0, 0], spare[2], 20], dtype=np.int32)
    # child not empty; out of range; child that is a parent; page in use; no such page
    st = pages.fork([], bt, sl, ref, [0, 9, 3, 1, 0, 0], [1, 2, 2, 2, 3, 4], new)
    assert st == pages.REFUSED and (new == -1).all()
    assert all(np.array_equal(a, b) for a, b in zip(state, (bt, sl, ref)))


def test_compaction_keeps_every_row_and_count():
    r = np.random.default_rng(5)
    bt, sl, ref, spare = _pool(r, 40, 4, 5, [70, 3, 17, 0])
    ref[spare[0]] = 2                                  # held outside the tables
    cache = r.integers(0, 1 << 30, (40, 3))
    rows = [cache[bt[i, :-(-int(sl[i]) // 16)]].copy() for i in range(4)]
    outside = cache[spare[0]].copy()
    counts = sorted(ref[ref > 0])
    st, page_map, n = pages.compact([cache], bt, ref)
    assert st == 0 and n == 9 and (ref[:9] > 0).all() and (ref[9:] == 0).all() and sorted(ref[:9]) == counts
    for i in range(4):
        assert np.array_equal(cache[bt[i, :-(-int(sl[i]) // 16)]], rows[i])
    assert np.array_equal(cache[page_map[spare[0]]], outside) and (bt < 9).all()
