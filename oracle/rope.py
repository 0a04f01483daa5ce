"""Float64 CPU oracle for rotary positions with several axes and the cache write
(TEST INFRASTRUCTURE ONLY).

Pair i of a row's rotated features (x, y) becomes (x c - y s, y c + x s), with c and
s the i-th cosine and sine of the table's row at the token's position on that pair's
axis.  Key and value rows go to page slot // 16, slot % 16; tokens with a negative
slot, or one past the pool, write no cache row; a token whose position lies outside
the table on any axis writes nothing at all."""
from __future__ import annotations

import numpy as np

from .cache_write import e4m3fn_encode
from .paged_attention import PAGE_SIZE


def rotate(x, positions, table, pair_axis, neighbours, dtype=np.float64):
    """Rows [T, H, D] rotated; every operation in `dtype`.  positions [axes, T]."""
    x = np.asarray(x, dtype=dtype)
    out, n = x.copy(), table.shape[1] // 2
    for i in range(n):
        u, v = (2 * i, 2 * i + 1) if neighbours else (i, i + n)
        p = positions[0 if pair_axis is None else pair_axis[i]]
        c, s = table[p, i].astype(dtype)[:, None], table[p, n + i].astype(dtype)[:, None]
        out[:, :, u] = x[:, :, u] * c - x[:, :, v] * s
        out[:, :, v] = x[:, :, v] * c + x[:, :, u] * s
    return out


def bf16_bits(x):
    """float32 values -> bf16 bit patterns, round to nearest even (finite values)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def rope_cache_write(query, key, value, positions, table, pair_axis, neighbours, slots, k_cache, v_cache, k_scale,
                     v_scale, query_out, key_out=None):
    """The call bit by bit, its arithmetic in fp32 as defined: (query_out, key_out, k_cache, v_cache), new arrays.
    query / key / value float32 (bf16 values); caches and outputs uint16 bf16 patterns (caches of uint8: e4m3fn codes)."""
    positions = np.atleast_2d(positions)
    ok = ((positions >= 0) & (positions < table.shape[0])).all(0)
    safe = np.clip(positions, 0, table.shape[0] - 1)
    q = rotate(query, safe, table, pair_axis, neighbours, np.float32)
    k = rotate(key, safe, table, pair_axis, neighbours, np.float32)
    query_out, kc, vc = query_out.copy(), k_cache.copy(), v_cache.copy()
    query_out[ok] = bf16_bits(q[ok])
    if key_out is not None:
        key_out = key_out.copy()
        key_out[ok] = bf16_bits(k[ok])
    for t, s in enumerate(slots):
        if not ok[t] or s < 0 or s >= k_cache.shape[0] * PAGE_SIZE:
            continue
        for cache, row, scale in ((kc, k[t], k_scale), (vc, np.asarray(value[t], np.float32), v_scale)):
            if cache.dtype == np.uint8:
                with np.errstate(over="ignore"):
                    cache[s // PAGE_SIZE, s % PAGE_SIZE] = e4m3fn_encode((row / np.float32(scale)).astype(np.float64))
            else:
                cache[s // PAGE_SIZE, s % PAGE_SIZE] = bf16_bits(row)
    return query_out, key_out, kc, vc
