"""Float64 CPU oracle of decode attention over windows with first tokens that stay
visible and over batches that share prefixes (TEST INFRASTRUCTURE ONLY).

A query token at position p sees the keys j <= p with, where window > 0, j > p - window
or j < first.  Only the keys that some query token of a sequence sees are gathered, so
what the other slots hold cannot matter.  Sharing pages changes no result: the shared
batch's oracle is the same function on the same block tables."""
from __future__ import annotations

import numpy as np

from .paged_attention import PAGE_SIZE


def visible(p, n, window, first):
    """Truth values of the keys 0 .. n - 1 for position p."""
    j = np.arange(n)
    return (j <= p) & ((window <= 0) | (j > p - window) | (j < first))


def decode(q, k, v, block_tables, seq_lens, qsl, scale, window=0, first=0, sinks=None):
    """q float64 [T, Hq, D]; k, v float64 [NB, 16, Hkv, D].  Returns (out, lse, spread): spread is the attention of
    |v| (what roundings of the weights can move), NaN in rows of no sequence."""
    T, hq, d = q.shape
    hkv = k.shape[2]
    g = hq // hkv
    sc = float(np.float32(scale))
    out, spread = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan)
    lse = np.full((T, hq), np.nan)
    qsl = np.arange(len(seq_lens) + 1) if qsl is None else np.asarray(qsl)
    for i, L in enumerate(np.asarray(seq_lens).tolist()):
        qn = int(qsl[i + 1] - qsl[i])
        masks = [visible(L - qn + r, L, window, first) for r in range(qn)]
        seen = np.flatnonzero(np.any(masks, axis=0)) if qn and L else np.zeros(0, int)
        page = np.asarray(block_tables)[i][seen // PAGE_SIZE].astype(np.int64)
        ki, vi = k[page, seen % PAGE_SIZE], v[page, seen % PAGE_SIZE]
        for r in range(qn):
            t = int(qsl[i]) + r
            s = sc * np.einsum("hgd,jhd->hgj", q[t].reshape(hkv, g, d), ki)
            s = np.where(masks[r][seen], s, -np.inf)
            sink = np.full((hkv, g, 1), -np.inf) if sinks is None else \
                np.asarray(sinks, np.float32).astype(np.float64).reshape(hkv, g, 1)
            z = np.concatenate([s, sink], -1)
            m = z.max(-1, keepdims=True)
            m0 = np.where(np.isneginf(m), 0.0, m)
            w = np.exp(z - m0)
            total = w.sum(-1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[t] = (m0 + np.log(total)).reshape(hq)
            p = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)[..., :-1]
            p = np.where(np.isnan(total), np.nan, p)
            # a key that the row does not see cannot reach it, whatever it holds
            val = np.where(masks[r][seen][:, None, None], vi, 0.0)
            out[t] = np.einsum("hgj,jhd->hgd", p, val).reshape(hq, d)
            spread[t] = np.einsum("hgj,jhd->hgd", p, np.abs(val)).reshape(hq, d)
    return out, lse, spread
