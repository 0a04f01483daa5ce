"""Seeded batches for the tests of decode calls over walks with a hole, and the bounds
their results are held to."""
import numpy as np
import torch

from oracle import e4m3fn_to_float64, walk
from paged_kv_decode_06_gb300 import binding


class Batch:
    """Sequences over a paged cache of permuted pages.  groups: (first sequence of each and the end, tokens shared):
    the sequences of a group hold the same pages for their shared whole pages."""

    def __init__(self, lens, qlens=None, hq=8, hkv=2, d=128, kv="bf16", seed=0, sinks=False, groups=None, extra=3,
                 pad_rows=0, scale=None, tokens=False, holes=False):
        r = np.random.default_rng(seed)
        self.lens = np.array(lens, dtype=np.int32)
        self.qlens = np.ones(len(lens), dtype=np.int64) if qlens is None else np.array(qlens)
        self.qsl = None if qlens is None else np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.runs = 1 if qlens is None else max(1, int(self.qlens.max()))
        self.hq, self.hkv, self.d, self.kv = hq, hkv, d, kv
        self.scale = d ** -0.5 if scale is None else scale
        self.ks, self.vs = (0.03, 0.02) if kv == "fp8" else (1.0, 1.0)
        n = -(-np.maximum(self.lens.astype(np.int64), 0) // 16)
        width = max(1, int(n.max()))
        nb = int(n.sum()) + extra
        order = iter(r.permutation(nb).tolist())
        self.bt = np.full((len(lens), width), -1, dtype=np.int32)
        heads = [0] * len(lens)
        self.groups = groups
        if groups is not None:
            for a, b, s in zip(groups[0], groups[0][1:], groups[1]):
                pages = [next(order) for _ in range(s // 16)]
                for i in range(a, b):
                    k = min(len(pages), int(n[i]))
                    self.bt[i, :k] = pages[:k]
                    heads[i] = k
        for i in range(len(lens)):
            for j in range(heads[i], int(n[i])):
                self.bt[i, j] = next(order)
        shape = (nb, 16, hkv, d)
        t = int(self.qlens.sum()) + pad_rows
        self.q = torch.from_numpy(r.standard_normal((t, hq, d)).astype(np.float32)).to(torch.bfloat16)
        if kv == "bf16":
            self.k, self.v = (torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)
                              for _ in range(2))
        else:
            # codes of normal rows of unit variance; no NaN code
            self.k, self.v = (torch.from_numpy(np.clip(r.standard_normal(shape) / s, -448, 448).astype(np.float32)).to(
                torch.float8_e4m3fn).view(torch.uint8) for s in (self.ks, self.vs))
        self.tk = self.tv = None
        if tokens:
            self.tk, self.tv = (torch.from_numpy(np.exp(r.standard_normal((nb, hkv, 16)) * 0.3).astype(np.float32))
                                for _ in range(2))
        self.sinks = r.standard_normal(hq).astype(np.float32) if sinks else None

    def values(self):
        """float64 keys and values of the whole pool."""
        if self.kv == "bf16":
            return self.k.double().numpy(), self.v.double().numpy()
        k = e4m3fn_to_float64(self.k.numpy()) * float(np.float32(self.ks))
        v = e4m3fn_to_float64(self.v.numpy()) * float(np.float32(self.vs))
        if self.tk is not None:
            k = k * self.tk.double().numpy().transpose(0, 2, 1)[..., None]
            v = v * self.tv.double().numpy().transpose(0, 2, 1)[..., None]
        return k, v

    def on_gpu(self):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.dsinks = None if self.sinks is None else c(self.sinks)
        self.dtok = (None, None) if self.tk is None else (self.tk.cuda(), self.tv.cuda())
        return [self.q.cuda(), self.k.cuda(), self.v.cuda(), c(self.bt), c(self.lens),
                None if self.qsl is None else c(self.qsl)]

    def options(self, **kw):
        return binding.make_options(sinks=self.dsinks, k_token_scales=self.dtok[0], v_token_scales=self.dtok[1], **kw)

    def buffers(self):
        return (torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full(self.q.shape[:2], 7.0, device="cuda"))

    def want(self, window=0, first=0):
        k, v = self.values()
        return walk.decode(self.q.double().numpy(), k, v, self.bt, self.lens, self.qsl, self.scale, window, first,
                           self.sinks)

    def check(self, out, lse, window=0, first=0, status=0):
        """Every row within the sum of the roundings on the way.  With A = sum_j p_j |v_j| of the row and feature:
        output to bf16 2^-8 |out|; weights rounded to bf16 2^-8 A (f16 for fp8 caches: 2^-11 A and 2^-25 of the largest
        weight for N small ones); N-term fp32 sums (weights, outputs, merges) N 2^-23 A; exponentials 2^-21 A; scores,
        fp32 sums of D products and three factors, ds = (D + 8) 2^-24 scale sum_d |q_d| max|k| (and D 2^-25 max|k| for
        query elements in f16), which move a weight relative to another by 2 ds."""
        assert binding.paged_attn_device_status() == status
        wo, wl, spread = self.want(window, first)
        go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        k, v = self.values()
        kmax, vmax = np.nanmax(np.abs(np.where(np.isinf(k), 0, k))), np.nanmax(np.abs(np.where(np.isinf(v), 0, v)))
        n = max(1, int(self.lens.max()))
        fill = np.arange(len(wl)) >= self.qlens.sum()
        assert (go[fill] == 7).all() and (gl[fill] == 7).all()      # rows of no sequence stay as they were
        go, gl, wo, wl, spread = go[~fill], gl[~fill], wo[~fill], wl[~fill], spread[~fill]
        aq = np.abs(self.q.double().numpy())[~fill].sum(-1)
        ds = abs(self.scale) * kmax * (aq * (self.d + 8) * 2.0 ** -24 + (self.d * 2.0 ** -25 if self.kv == "fp8" else 0))
        low = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11
        rel = low + n * 2.0 ** -23 + 2.0 ** -21 + 2 * ds
        tol = 2.0 ** -8 * np.abs(wo) + rel[..., None] * spread
        if self.kv == "fp8":
            tol = tol + n * 2.0 ** -25 * vmax
        tol = tol * (1 + 2.0 ** -6) + 2.0 ** -126                   # products of the terms; bf16's smallest
        assert (np.isnan(go) == np.isnan(wo)).all() and (np.isnan(gl) == np.isnan(wl)).all()
        ok = ~np.isnan(wo)
        assert (np.abs(go - wo)[ok] <= tol[ok]).all(), float((np.abs(go - wo) - tol)[ok].max())
        dead = np.isneginf(wl)
        assert (gl[dead] == -np.inf).all()
        live = ~dead & ~np.isnan(wl)
        lt = ds + n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(np.where(live, wl, 0)))
        assert (np.abs(gl - wl)[live] <= lt[live]).all(), float((np.abs(gl - wl) - lt)[live].max())
