"""Float64 CPU oracle of the 4-bit paged KV cache (TEST INFRASTRUCTURE ONLY).

The format: e2m1 codes packed two a byte (the even feature in the low nibble),
one e4m3fn scale code for 16 consecutive features of a cached row, one fp32
scale a tensor; value = e2m1 * e4m3 * scale.

``write_rows`` follows the entry point's definition: S = e4m3fn(amax / (6 s)),
codes e2m1(x / (S s)), where 6 s and S s are fp32 products and both quotients
IEEE fp32 quotients; round to nearest even, saturating; S = 0 stores codes 0, a
NaN in the group stores the NaN as S and codes 0.
"""
from __future__ import annotations

import numpy as np

from .cache_write import e4m3fn_encode
from .paged_attention import PAGE_SIZE, bf16_bits_to_float64, e4m3fn_to_float64

# sign, two exponent bits (bias 1), one mantissa bit
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP = 16


def e2m1_to_float64(codes: np.ndarray) -> np.ndarray:
    v = E2M1_VALUES[codes & 7]
    return np.where(codes & 8, -v, v)


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Nearest e2m1 code, ties to the even code, saturating to +-6; the sign bit is copied."""
    a = np.minimum(np.abs(x), 6.0)
    hi = np.searchsorted(E2M1_VALUES, a, side="left")
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - E2M1_VALUES[lo], E2M1_VALUES[hi] - a
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def quantise_rows(bits: np.ndarray, scale: float):
    """bf16 rows [..., D] -> (packed codes [..., D / 2], scale codes [..., D / 16])."""
    ts = np.float32(scale)
    x = bf16_bits_to_float64(bits).astype(np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)                               # NaN if the group holds one
        s = e4m3fn_encode((amax / (np.float32(6) * ts)).astype(np.float64))
        d = (e4m3fn_to_float64(s).astype(np.float32) * ts)[..., None]
        y = g / d
    live = d > 0
    code = np.where(live, e2m1_encode(np.where(live, y, np.float32(0)).astype(np.float64)), 0).astype(np.uint8)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def dequantise_rows(codes: np.ndarray, scales: np.ndarray, scale: float) -> np.ndarray:
    """float64 values of packed codes [..., D / 2] with scale codes [..., D / 16]."""
    x = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    x[..., 0::2] = e2m1_to_float64(codes & 15)
    x[..., 1::2] = e2m1_to_float64(codes >> 4)
    with np.errstate(invalid="ignore"):
        return x * np.repeat(e4m3fn_to_float64(scales), GROUP, axis=-1) * float(np.float32(scale))


def write_rows(bits, slots, codes, scales, scale):
    """(codes [NB, 16, H, D / 2], scales [NB, H, 16, D / 16]) after writing rows at their slots."""
    codes, scales = codes.copy(), scales.copy()
    c, s = quantise_rows(bits, scale)
    for t, slot in enumerate(slots):
        if 0 <= slot < PAGE_SIZE * codes.shape[0]:
            codes[slot // PAGE_SIZE, slot % PAGE_SIZE] = c[t]
            scales[slot // PAGE_SIZE, :, slot % PAGE_SIZE] = s[t]
    return codes, scales


def read_rows(slots, codes, scales, scale, before):
    """float64 rows [T, H, D]: the values at the slots, `before` where a slot is negative or past the pool."""
    out = np.array(before, dtype=np.float64)
    for t, slot in enumerate(slots):
        if 0 <= slot < PAGE_SIZE * codes.shape[0]:
            p, o = slot // PAGE_SIZE, slot % PAGE_SIZE
            out[t] = dequantise_rows(codes[p, o], scales[p, :, o], scale)
    return out


def decode(q, codes, scales, block_tables, seq_lens, query_start_loc, scale, k_scale, v_scale, window=0, sinks=None):
    """out, lse in float64 of decode attention over a 4-bit cache.

    q float64 [T, Hq, D]; codes = (K, V) [NB, 16, Hkv, D / 2]; scales = (K, V)
    [NB, Hkv, 16, D / 16].  A row that sees no key has out 0 and lse -inf (its
    sink's logit with sinks); rows of no sequence are NaN."""
    T, Hq, D = q.shape
    Hkv = codes[0].shape[2]
    G = Hq // Hkv
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    for i, L in enumerate(map(int, seq_lens)):
        t0, t1 = map(int, query_start_loc[i:i + 2]) if query_start_loc is not None else (i, i + 1)
        if t1 <= t0:
            continue
        j = np.arange(max(L, 0))
        page, off = block_tables[i][j // PAGE_SIZE], j % PAGE_SIZE
        k = dequantise_rows(codes[0][page, off], scales[0][page, :, off], k_scale)      # [L, Hkv, D]
        v = dequantise_rows(codes[1][page, off], scales[1][page, :, off], v_scale)
        for t in range(t0, t1):
            pos = L - (t1 - t0) + (t - t0)
            seen = (j <= pos) & ((j > pos - window) if window > 0 else True)
            for h in range(Hq):
                s = scale * (k[seen, h // G] @ q[t, h])
                if sinks is not None:
                    s = np.append(s, sinks[h])
                if s.size == 0:
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                m = s.max()
                p = np.exp(s - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                out[t, h] = p[:seen.sum()] @ v[seen, h // G]
    return out, lse


def decode_with_bounds(q, codes, scales, block_tables, seq_lens, query_start_loc, scale, k_scale, v_scale, window=0,
                       sinks=None):
    """out, lse as ``decode`` and how far an evaluation of the kernel's roundings may be from each.

    Per row of n keys with weights p_j (sink included in the normaliser), A = sum_j p_j |v_j| a feature:
      * a score is off by ds_j: fp32 sums of D products, (D + 4) 2^-24 of scale sum |q k|; query elements in
        f16, 2^-25 of the row's largest each; the fp32 factor, product and maximum, 2^-21 (|s_j| + |s_max|);
      * weights are off by delta = max ds_j + 2^-21 (the exponential) relative, in the sum and in the output;
      * weights are rounded to f16 for the output: 2^-11 relative, 2^-25 of the row's largest weight where
        that is more (a warp's largest weight is at least 1 in its own units);
      * fp32 sums: c = n / 16 + 1000 roundings of 2^-23 (tensor-core sums of 16 keys; pieces, warps, merge),
        in the sum and in the output;
      * one bf16 rounding of the output, 2^-8."""
    out, lse = decode(q, codes, scales, block_tables, seq_lens, query_start_loc, scale, k_scale, v_scale, window, sinks)
    T, Hq, D = q.shape
    G = Hq // codes[0].shape[2]
    tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    for i, L in enumerate(map(int, seq_lens)):
        t0, t1 = map(int, query_start_loc[i:i + 2]) if query_start_loc is not None else (i, i + 1)
        if t1 <= t0 or L <= 0:
            continue
        j = np.arange(L)
        page, off = block_tables[i][j // PAGE_SIZE], j % PAGE_SIZE
        k = dequantise_rows(codes[0][page, off], scales[0][page, :, off], k_scale)
        v = np.abs(dequantise_rows(codes[1][page, off], scales[1][page, :, off], v_scale))
        for t in range(t0, t1):
            pos = L - (t1 - t0) + (t - t0)
            seen = (j <= pos) & ((j > pos - window) if window > 0 else True)
            n = int(seen.sum())
            for h in range(Hq):
                if n == 0:
                    continue
                kh, row = k[seen, h // G], q[t, h]
                s = scale * (kh @ row)
                p = np.exp(s - lse[t, h])
                top = max(np.abs(s).max(), abs(float(sinks[h])) if sinks is not None else 0.0)
                ds = abs(scale) * ((D + 4) * 2.0 ** -24 * (np.abs(kh) @ np.abs(row)) +
                                   2.0 ** -25 * np.abs(row).max() * np.abs(kh).sum(-1)) + 2.0 ** -20 * top
                delta, c = ds.max() + 2.0 ** -21, (n / 16 + 1000) * 2.0 ** -23
                vh = v[seen, h // G]
                err = (2.0 ** -11 + 2 * delta + 2 * c) * (p @ vh) + 2.0 ** -25 * p.max() * vh.sum(0)
                tol[t, h] = err + 2.0 ** -8 * (np.abs(out[t, h]) + err)
                tol_lse[t, h] = delta + c + 2.0 ** -21 + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, tol, tol_lse
