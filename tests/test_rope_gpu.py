"""paged_attn_rope_cache_write against its definition, bit by bit: the arithmetic is
one fp32 product, sum and rounding at a time, so every stored bit is determined."""
import numpy as np
import pytest
import torch

from oracle import rope
from paged_kv_decode_06_gb300 import binding

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _table(rows, rot, theta=10000.0):
    ang = np.arange(rows)[:, None] * theta ** (-2.0 * np.arange(rot // 2) / rot)[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _bits(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16).cpu().numpy().view(
        np.uint8 if x.element_size() == 1 else np.uint16)


class Case:
    def __init__(self, t, hq, hkv, d, rot, axes, kv="bf16", neighbours=False, axis="blocks", nb=None, rows=300, seed=0,
                 strided=False, bad=False):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.nb = nb or t // 16 + 3
        self.neighbours = neighbours
        mk = lambda h: torch.randn(t, h + (1 if strided else 0), d + (8 if strided else 0), generator=g).to(bf).cuda()
        cut = lambda x, h: x[:, :h, :d]
        self.q, self.k, self.v = (cut(mk(h), h) for h in (hq, hkv, hkv))
        self.pos = r.integers(0, rows, (axes, t)).astype(np.int32)
        self.slots = r.permutation(self.nb * 16)[:t].astype(np.int32)
        self.slots[r.random(t) < 0.1] = -1
        if bad and t > 3:
            self.pos[axes - 1, 0], self.pos[0, t - 1] = rows, -1
            self.slots[1] = self.nb * 16
        self.table = _table(rows, rot)
        n = rot // 2
        self.axis = None if axes == 1 else [i % axes for i in range(n)] if axis == "turns" else \
            [min(i * axes // n, axes - 1) for i in range(n)]
        dt = bf if kv == "bf16" else torch.uint8
        mkc = lambda: (torch.randint(0, 120, (self.nb, 16, hkv + (1 if strided else 0), d), generator=g).to(dt).cuda())[:, :, :hkv]
        self.kc, self.vc = mkc(), mkc()
        self.ks, self.vs = (0.05, 0.031) if kv == "fp8" else (1.0, 1.0)

    def run(self, key_out=False, in_place=False, **kw):
        dev = lambda x: torch.from_numpy(x).cuda()
        self.q0, self.k0 = self.q.clone(), self.k.clone()
        self.kc0, self.vc0 = self.kc.clone(), self.vc.clone()
        qo = self.q if in_place else torch.full(self.q.shape, 3.0, dtype=bf, device="cuda")
        ko = (self.k if in_place else torch.full(self.k.shape, 3.0, dtype=bf, device="cuda")) if key_out else None
        self.qo0, self.ko0 = qo.clone(), None if ko is None else ko.clone()
        pos = self.pos[0] if self.axis is None else self.pos
        got = binding.paged_attn_rope_cache_write(self.q, self.k, self.v, dev(pos), dev(self.table), dev(self.slots),
                                                  self.kc, self.vc, self.axis, self.neighbours, self.ks, self.vs, qo,
                                                  ko, **kw)
        assert got is qo
        torch.cuda.synchronize()
        return qo, ko

    def check(self, qo, ko, status=0):
        assert binding.paged_attn_device_status() == status
        want = rope.rope_cache_write(self.q0.float().cpu().numpy(), self.k0.float().cpu().numpy(),
                                     self.v.float().cpu().numpy(), self.pos, self.table, self.axis, self.neighbours,
                                     self.slots, _bits(self.kc0), _bits(self.vc0), self.ks, self.vs, _bits(self.qo0),
                                     None if ko is None else _bits(self.ko0))
        for name, a, b in (("query", qo, want[0]), ("key", ko, want[1]), ("k cache", self.kc, want[2]),
                           ("v cache", self.vc, want[3])):
            if a is not None:
                assert (_bits(a) == b).all(), name


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,rot,axes,axis", [
    (1, 1, 1, 16, 16, 1, "blocks"), (3, 8, 2, 64, 64, 3, "turns"), (17, 5, 5, 128, 128, 3, "blocks"),
    (33, 7, 1, 96, 48, 2, "turns"), (5, 2, 2, 80, 20, 3, "blocks"), (64, 12, 3, 48, 12, 1, "blocks"),
    (130, 4, 2, 256, 64, 2, "blocks"), (9, 3, 1, 512, 512, 3, "turns"), (2, 70, 9, 32, 4, 2, "turns")])
def test_bit_by_bit(t, hq, hkv, d, rot, axes, axis, neighbours, kv):
    c = Case(t, hq, hkv, d, rot, axes, kv, neighbours, axis)
    c.check(*c.run(key_out=True))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_many_tokens(kv):
    c = Case(3000, 32, 8, 128, 128, 3, kv, axis="turns", rows=5000)
    c.check(*c.run())
    c = Case(5000, 6, 3, 40, 12, 3, kv) if kv == "bf16" else Case(5000, 6, 3, 48, 12, 3, kv)
    c.check(*c.run(key_out=True))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("rot", [64, 24])
def test_strided_in_place(kv, rot):
    c = Case(40, 6, 3, 64, rot, 3, kv, strided=True)
    c.check(*c.run(key_out=True, in_place=True))


def test_bad_positions_and_slots_write_nothing():
    c = Case(50, 4, 2, 64, 64, 3, bad=True)
    c.check(*c.run(key_out=True), status=binding.STATUS_POSITION | binding.STATUS_PAGE_RANGE)


def test_special_values():
    """NaN and infinities stay in their own pairs; an fp8 cache saturates infinities and keeps NaN's code."""
    c = Case(8, 2, 2, 64, 64, 1)
    c.q[0, 0, 3], c.k[1, 1, 5], c.v[2, 0, 7] = float("nan"), float("inf"), float("-inf")
    qo, _ = c.run()
    bad = torch.isnan(qo) | torch.isinf(qo)
    assert bad[0, 0, 3] and bad[0, 0, 35] and int(bad.sum()) == 2
    assert int((~torch.isfinite(c.kc)).sum()) in (0, 2) and int(torch.isinf(c.vc).sum()) in (0, 1)


def test_other_stream_and_graph():
    c = Case(20, 4, 2, 64, 64, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.check(*c.run(stream=s))
    c = Case(20, 4, 2, 64, 64, 3, seed=5)
    dev = lambda x: torch.from_numpy(x).cuda()
    pos, tab, slots = dev(c.pos), dev(c.table), dev(c.slots)
    qo = torch.zeros_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.paged_attn_rope_cache_write(c.q, c.k, c.v, pos, tab, slots, c.kc, c.vc, c.axis, query_out=qo)
    c.q.copy_(torch.randn(c.q.shape).to(bf))
    c.q0, c.k0, c.kc0, c.vc0, c.qo0 = c.q.clone(), c.k.clone(), c.kc.clone(), c.vc.clone(), qo.clone()
    g.replay()
    torch.cuda.synchronize()
    c.check(qo, None)


def test_table_rows_past_32_bit_offsets():
    """A position whose row lies more than 2^31 elements into the table."""
    rows = 35_000_000
    tab = torch.zeros(rows, 64, device="cuda")
    tab[-1] = torch.from_numpy(_table(77, 64)[76]).cuda()
    c = Case(4, 2, 1, 64, 64, 1)
    pos = torch.full((4,), rows - 1, dtype=torch.int32, device="cuda")
    qo = binding.paged_attn_rope_cache_write(c.q, c.k, c.v, pos, tab, torch.from_numpy(c.slots).cuda(), c.kc, c.vc)
    want = rope.bf16_bits(rope.rotate(c.q.float().cpu().numpy(), np.full((1, 4), 76), _table(77, 64), None, False, np.float32))
    assert (_bits(qo) == want).all()
