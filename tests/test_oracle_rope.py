"""Pins of the rotary oracle, and the binding's pair-axis helper (no GPU)."""
import numpy as np
import pytest

from oracle import rope
from paged_kv_decode_06_gb300 import binding


def _table(rows, rot, theta=10000.0):
    ang = np.arange(rows)[:, None] * theta ** (-2.0 * np.arange(rot // 2) / rot)[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotation_is_a_complex_product(neighbours):
    r = np.random.default_rng(0)
    t, rot, d = 7, 12, 20
    x, tab = r.standard_normal((t, 3, d)), _table(50, rot)
    pos = r.integers(0, 50, (2, t))
    axis = [i % 2 for i in range(rot // 2)]
    y = rope.rotate(x, pos, tab, axis, neighbours)
    z = lambda a: a[..., 0:rot:2] + 1j * a[..., 1:rot:2] if neighbours else a[..., :rot // 2] + 1j * a[..., rot // 2:rot]
    ang = np.stack([np.arctan2(tab[pos[a], 6 + i], tab[pos[a], i]) for i, a in enumerate(axis)], 1)
    assert np.allclose(z(y), z(x) * np.exp(1j * ang)[:, None], atol=1e-12)
    assert (y[..., rot:] == x[..., rot:]).all()


def test_products_depend_on_the_distance_alone():
    r = np.random.default_rng(1)
    q, k, tab = r.standard_normal((1, 1, 16)), r.standard_normal((1, 1, 16)), _table(200, 16)
    dot = lambda a, b: float((rope.rotate(q, np.array([[a]]), tab, None, False) *
                              rope.rotate(k, np.array([[b]]), tab, None, False)).sum())
    assert abs(dot(30, 11) - dot(130, 111)) < 1e-10 and abs(dot(30, 11) - dot(30, 12)) > 1e-3


def test_position_zero_changes_nothing_and_norms_stay():
    r = np.random.default_rng(2)
    x, tab = r.standard_normal((4, 2, 8)), _table(9, 8)
    assert (rope.rotate(x, np.zeros((1, 4), int), tab, None, True) == x).all()
    y = rope.rotate(x, np.array([[8, 1, 3, 5]]), tab, None, True)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))


def test_bf16_rounding_goes_to_even():
    x = np.array([1.0, 1.00390625, 1.01171875, -1.00390625, 1.005, 0.0], np.float32)
    assert [hex(v) for v in rope.bf16_bits(x)] == ["0x3f80", "0x3f80", "0x3f82", "0xbf80", "0x3f81", "0x0"]


def test_writes_leave_padding_and_bad_positions_alone():
    r = np.random.default_rng(3)
    q, k, v = (r.standard_normal((4, 1, 8)).astype(np.float32) for _ in range(3))
    kc = np.full((2, 16, 1, 8), 7, np.uint16)
    qo = np.full((4, 1, 8), 9, np.uint16)
    out, _, kn, vn = rope.rope_cache_write(q, k, v, np.array([1, 2, 3, 99]), _table(9, 8), None, False,
                                           np.array([5, -1, 64, 6]), kc, kc, 1.0, 1.0, qo)
    assert (out[3] == 9).all() and not (out[:3] == 9).any(axis=(1, 2)).all()
    changed = np.argwhere((kn != 7).any(-1))
    assert changed.tolist() == [[0, 5, 0]] and (vn[0, 5, 0] == rope.bf16_bits(v[0, 0])).all()


def test_pair_axes():
    assert binding.rope_pair_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert binding.rope_pair_axes([4, 2, 2], in_turn=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert binding.rope_pair_axes([5]) == [0] * 5
