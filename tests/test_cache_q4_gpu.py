"""paged_attn_cache_write_q4 and _read_q4 against the oracle: codes and scales
bit for bit (the same fp32 products and IEEE quotients), values read back after
one fp32 and one bf16 rounding."""
import threading

import numpy as np
import pytest
import torch

from oracle import cache_q4
from paged_kv_decode_06_gb300 import binding

pytestmark = pytest.mark.gpu

KS, VS = 0.05, 0.013


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _cache(NB, Hkv, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda hi, *s: torch.randint(0, hi, s, dtype=torch.uint8, device="cuda", generator=g)
    return (mk(256, NB, 16, Hkv, D // 2), mk(256, NB, 16, Hkv, D // 2),
            mk(127, NB, Hkv, 16, D // 16), mk(127, NB, Hkv, 16, D // 16))


def _rows(T, Hkv, D, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda: (torch.randn(T, Hkv, D, device="cuda", generator=g) *
                 torch.exp(spread * torch.randn(T, Hkv, D // 16, 1, device="cuda", generator=g)).expand(
                     T, Hkv, D // 16, 16).reshape(T, Hkv, D)).to(torch.bfloat16)
    return f(), f()


def _check(key, val, slots, cache, ks=KS, vs=VS, status=0):
    """Write, compare the whole cache; read back, compare within the two roundings."""
    kc, vc, ksc, vsc = cache
    before = [t.cpu().numpy().copy() for t in cache]
    sl = torch.as_tensor(np.asarray(slots, dtype=np.int32)).cuda()
    binding.paged_attn_cache_write_q4(key, val, sl, kc, vc, ksc, vsc, ks, vs)
    assert binding.paged_attn_device_status() == status
    for x, c, s, ts, b0, b1 in ((key, kc, ksc, ks, before[0], before[2]), (val, vc, vsc, vs, before[1], before[3])):
        ec, es = cache_q4.write_rows(_bits(x), slots, b0, b1, ts)
        assert np.array_equal(s.cpu().numpy(), es)
        assert np.array_equal(c.cpu().numpy(), ec)
    ko, vo = torch.full_like(key, 7.0), torch.full_like(val, 7.0)
    binding.paged_attn_cache_read_q4(sl, kc, vc, ksc, vsc, ko, vo, ks, vs)
    assert binding.paged_attn_device_status() == status
    for o, c, s, ts in ((ko, kc, ksc, ks), (vo, vc, vsc, vs)):
        want = cache_q4.read_rows(slots, c.cpu().numpy(), s.cpu().numpy(), ts, np.full(o.shape, 7.0))
        got = o.double().cpu().numpy()
        assert np.array_equal(np.isnan(want), np.isnan(got))
        # the fp32 product (2^-24 of the value), then bf16 (2^-8): 2^-8 (1 + 2^-24) + 2^-24 < 2^-8 + 2^-23;
        # below 2^-126 both have a fixed step (2^-149, 2^-133) and are off by half of it: 2^-150 + 2^-134 < 2^-133
        ok = np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133
        assert (ok | np.isnan(want)).all()


@pytest.mark.parametrize("T,Hkv,D,NB", [(1, 1, 16, 1), (1, 1, 64, 2), (37, 2, 128, 9), (500, 8, 128, 80),
                                        (77, 3, 48, 6), (150, 5, 80, 12), (45, 3, 512, 4), (3000, 8, 64, 200)])
def test_rows_bit_exact(T, Hkv, D, NB):
    key, val = _rows(T, Hkv, D, T + D)
    r = np.random.default_rng(T)
    slots = r.permutation(NB * 16)[:T].astype(np.int32)
    slots[r.random(T) < 0.1] = -1
    _check(key, val, slots, _cache(NB, Hkv, D, T))


@pytest.mark.parametrize("ks,vs", [(1.0, 1.0), (0.05, 0.07), (1e-30, 3e30), (2.0 ** -149, 2.0 ** -126), (1e38, 5e37)])
def test_extreme_tensor_scales(ks, vs):
    """Group scales that vanish, are subnormal or saturate, and 6 s past the fp32 range."""
    key, val = _rows(64, 2, 64, 5, spread=8.0)
    _check(key, val, np.arange(64, dtype=np.int32)[::-1].copy(), _cache(4, 2, 64, 1), ks, vs)


def test_special_values():
    key, val = _rows(8, 1, 64, 6)
    key[0], key[1] = 0.0, -0.0
    key[2, 0, 3] = float("nan")
    key[3, 0, 17], key[3, 0, 40] = float("inf"), -float("inf")
    key[4] = 3.3e38
    val[5] = 1e-40
    val[6, 0, 5], val[6, 0, 6] = float("nan"), float("inf")
    val[7] = -1.0
    _check(key, val, np.arange(8, dtype=np.int32), _cache(1, 1, 64, 2))


def test_every_code_and_tie():
    """Rows of exact code midpoints (ties to even) and codes at every scale exponent."""
    grid = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -6.0])
    x = torch.stack([grid * 2.0 ** e for e in range(-14, 9)] + [-grid * 2.0 ** e for e in range(-14, 9)])
    x = x.reshape(46, 1, 16).to(torch.bfloat16).cuda()
    _check(x, x.clone(), np.arange(46, dtype=np.int32), _cache(3, 1, 16, 3), 1.0, 0.5)


def test_strided_rows_caches_and_scales():
    T, Hkv, D, NB = 40, 3, 64, 5
    wide = torch.randn(T, 2, Hkv + 1, D + 8, device="cuda").to(torch.bfloat16)
    key, val = wide[:, 0, :Hkv, :D], wide[:, 1, 1:, :D]
    codes = torch.randint(0, 256, (NB, 2, 17, Hkv, D // 2 + 8), dtype=torch.uint8, device="cuda")
    sc = torch.randint(0, 127, (NB, 2, 16, Hkv, D // 16 + 3), dtype=torch.uint8, device="cuda")
    kc, vc = codes[:, 0, 1:, :, :D // 2], codes[:, 1, :16, :, 8:]
    ks, vs = sc[:, 0, :, :, :D // 16].transpose(1, 2), sc[:, 1, :, :, 3:].transpose(1, 2)
    rest = codes.clone(), sc.clone()
    slots = np.random.default_rng(0).permutation(NB * 16)[:T].astype(np.int32)
    _check(key, val, slots, (kc, vc, ks, vs))
    # nothing outside the views changed
    assert torch.equal(codes[:, 0, 0], rest[0][:, 0, 0]) and torch.equal(codes[:, 1, 16], rest[0][:, 1, 16])
    assert torch.equal(codes[:, 0, :, :, D // 2:], rest[0][:, 0, :, :, D // 2:])
    assert torch.equal(sc[:, 0, :, :, D // 16:], rest[1][:, 0, :, :, D // 16:])


def test_slot_past_the_pool_is_reported_and_skipped():
    key, val = _rows(4, 2, 32, 8)
    _check(key, val, np.array([3, 32, -5, 31], dtype=np.int32), _cache(2, 2, 32, 4),
           status=binding.STATUS_PAGE_RANGE)


def test_empty_call_and_float4_views():
    cache = _cache(2, 1, 32, 9)
    none = torch.empty(0, 1, 32, dtype=torch.bfloat16, device="cuda")
    binding.paged_attn_cache_write_q4(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), *cache)
    key, val = _rows(3, 1, 32, 9)
    slots = torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda")
    binding.paged_attn_cache_write_q4(key, val, slots, *cache, KS, VS)
    f8 = [t.view(torch.float8_e4m3fn) for t in cache[2:]]
    a = binding.paged_attn_cache_read_q4(slots, *cache, k_scale=KS, v_scale=VS)
    b = binding.paged_attn_cache_read_q4(slots, *cache[:2], *f8, k_scale=KS, v_scale=VS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_written_in_a_graph_on_another_stream():
    key, val = _rows(33, 2, 64, 10)
    cache = _cache(4, 2, 64, 11)
    slots = torch.arange(33, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.paged_attn_cache_write_q4(key, val, slots, *cache, KS, VS)
    key2, val2 = _rows(33, 2, 64, 12)
    key.copy_(key2)
    val.copy_(val2)
    slots.copy_(torch.arange(33, dtype=torch.int32).flip(0))
    want = [t.cpu().numpy() for t in cache]
    graph.replay()
    torch.cuda.synchronize()
    ec, es = cache_q4.write_rows(_bits(key2), np.arange(33)[::-1], want[0], want[2], KS)
    assert np.array_equal(cache[0].cpu().numpy(), ec) and np.array_equal(cache[2].cpu().numpy(), es)


def test_tensors_off_the_device_are_refused():
    key, val = _rows(2, 1, 32, 13)
    cache = _cache(1, 1, 32, 13)
    with pytest.raises(ValueError):
        binding.paged_attn_cache_write_q4(key.cpu(), val, torch.zeros(2, dtype=torch.int32, device="cuda"), *cache)


@pytest.mark.parametrize("T,Hkv,D", [(6, 2, 256), (2500, 8, 128), (5000, 3, 48), (20000, 8, 16)])
def test_rows_by_lane_groups(T, Hkv, D):
    """Calls that fill the device and calls that do not, rows of 2 to 32 chunks, warps past the last row."""
    key, val = _rows(T, Hkv, D, T + D)
    r = np.random.default_rng(T)
    NB = -(-T // 16) + 2
    slots = r.permutation(NB * 16)[:T].astype(np.int32)
    slots[r.random(T) < 0.05] = -1
    _check(key, val, slots, _cache(NB, Hkv, D, T))


def test_two_threads_with_tensors_of_one_layout():
    """Calls of the same types and shapes from two threads at once, each with its own tensors and stream."""
    work = []
    for seed in (1, 2):
        key, val = _rows(300, 2, 64, seed)
        cache = _cache(20, 2, 64, seed)
        slots = torch.randperm(320, device="cuda", dtype=torch.int32)[:300]
        want = [t.clone() for t in cache]
        binding.paged_attn_cache_write_q4(key, val, slots, *want, KS, VS)
        work.append((key, val, slots, cache, want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def run(key, val, slots, cache, want, stream):
        for _ in range(200):
            binding.paged_attn_cache_write_q4(key, val, slots, *cache, KS, VS, stream=stream)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for _, _, _, cache, want, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(cache, want))
