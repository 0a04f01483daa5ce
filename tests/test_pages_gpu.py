"""The page operations against their plain statement: contents, tables, counts
and lists bit for bit."""
import numpy as np
import pytest
import torch

from oracle import pages
from paged_kv_decode_06_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _caches(nb, kinds, seed=0):
    """Page tensors of several element types and layouts (views of larger tensors among them)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)
    make = {
        "bf16": lambda: byte(nb, 16, 3, 128).view(torch.bfloat16),
        "q4": lambda: byte(nb, 16, 2, 32),
        "scale": lambda: byte(nb, 1, 16, 4),
        "mla": lambda: byte(nb, 16, 1152).view(torch.bfloat16),
        "big": lambda: byte(nb, 16, 8, 256).view(torch.bfloat16),
        "flat": lambda: byte(nb, 20).view(torch.float32),
        "odd": lambda: byte(nb, 5, 7),
        "kv": lambda: byte(nb, 2, 16, 2, 64)[:, 1],                     # K and V side by side
        "padded": lambda: byte(nb, 16, 4, 80).view(torch.bfloat16)[:, :, 1:3, :32],
        "off": lambda: byte(nb, 16, 3, 41)[:, :, :, 1:38],              # byte-aligned runs
        "heads": lambda: byte(nb, 16, 4, 64).transpose(1, 2),
        "pages_inner": lambda: byte(16, nb, 2, 64).transpose(0, 1),
    }
    return [make[k]() for k in kinds]


ALL = ["bf16", "q4", "scale", "mla", "big", "flat", "odd", "kv", "padded", "off", "heads", "pages_inner"]


def _raw(c):
    """A host copy of a page tensor's bytes."""
    t = c.cpu().contiguous()
    return t.view(torch.uint8).numpy().reshape(t.shape[0], -1).copy()


def _same(caches, host):
    for c, h in zip(caches, host):
        assert np.array_equal(_raw(c), h)


@pytest.mark.parametrize("kinds", [[k] for k in ALL] + [ALL, ["q4", "scale"] * 60])
@pytest.mark.parametrize("nb,n", [(2, 1), (40, 13)])
def test_copy(kinds, nb, n):
    caches = _caches(nb, kinds)
    r = np.random.default_rng(n)
    perm = r.permutation(nb)
    src, dst = perm[r.integers(0, nb - n, n)].astype(np.int32), perm[nb - n:].astype(np.int32)
    if n > 5:
        src[2] = -1
        dst[4] = -7
        src[5] = dst[5]
    host = [_raw(c) for c in caches]
    binding.paged_attn_pages_copy(caches, _i32(src), _i32(dst))
    assert binding.paged_attn_device_status() == pages.copy(host, src, dst) == 0
    _same(caches, host)


def test_copy_views_leave_the_rest():
    base = torch.randint(0, 256, (9, 16, 4, 40), dtype=torch.uint8, device="cuda")
    keep = base.clone()
    binding.paged_attn_pages_copy([base[:, :, 1:3, 8:24]], _i32([0, 1]), _i32([5, 6]))
    torch.cuda.synchronize()
    want = keep.clone()
    want[5:7, :, 1:3, 8:24] = keep[0:2, :, 1:3, 8:24]
    assert torch.equal(base, want)


def test_copy_out_of_range_and_empty():
    caches = _caches(6, ["q4", "flat"])
    host = [_raw(c) for c in caches]
    binding.paged_attn_pages_copy(caches, _i32([0, 6, 2]), _i32([3, 1, 99]))
    assert binding.paged_attn_device_status() == pages.copy(host, [0, 6, 2], [3, 1, 99]) == binding.STATUS_PAGE_RANGE
    binding.paged_attn_pages_copy(caches, _i32([]), _i32([]))
    _same(caches, host)


def test_copy_many_pages():
    caches = _caches(3000, ["big", "q4"], 3)
    r = np.random.default_rng(3)
    perm = r.permutation(3000)
    src, dst = perm[:1500].astype(np.int32), perm[1500:].astype(np.int32)
    host = [_raw(c) for c in caches]
    binding.paged_attn_pages_copy(caches, _i32(src), _i32(dst))
    pages.copy(host, src, dst)
    _same(caches, host)


def _pool(r, nb, rows, lens, cols):
    order = r.permutation(nb)
    bt, ref, at = np.full((rows, cols), -1, dtype=np.int32), np.zeros(nb, dtype=np.int32), 0
    for i, n in enumerate(lens):
        k = -(-n // 16)
        bt[i, :k] = order[at:at + k]
        ref[order[at:at + k]] = 1
        at += k
    sl = np.zeros(rows, dtype=np.int32)
    sl[:len(lens)] = lens
    return bt, sl, ref, order[at:]


def _fork(caches, bt, sl, ref, par, chi, new, status=0):
    """Fork on both sides and compare everything; returns the device tensors."""
    host = [_raw(c) for c in caches]
    dev = [_i32(x) for x in (bt, sl, ref, par, chi, new)]
    binding.paged_attn_pages_fork(caches, *dev)
    assert binding.paged_attn_device_status() == pages.fork(host, bt, sl, ref, par, chi, new) == status
    for d, h in zip(dev, (bt, sl, ref, par, chi, new)):
        assert np.array_equal(d.cpu().numpy(), h)
    _same(caches, host)
    return dev


@pytest.mark.parametrize("rows,forks,hi", [(2, 1, 1), (8, 4, 50), (300, 290, 400), (2000, 900, 40)])
def test_fork_and_free(rows, forks, hi):
    r = np.random.default_rng(rows)
    lens = r.integers(1, hi + 1, rows - forks)
    need = int((-(-lens // 16)).sum())
    nb = need + forks + 3
    bt, sl, ref, spare = _pool(r, nb, rows, lens, -(-hi // 16))
    par = r.integers(0, rows - forks, forks).astype(np.int32)
    chi = (rows - forks + r.permutation(forks)).astype(np.int32)
    new = spare[:forks].astype(np.int32)
    par[forks // 2] = -1 if forks > 2 else par[forks // 2]
    ref0 = ref.copy()
    caches = _caches(nb, ["q4", "scale", "padded"], rows)
    dbt, dsl, dref, _, dchi, _ = _fork(caches, bt, sl, ref, par, chi, new)
    # free the children, one of them twice, and padding
    rows_ = np.concatenate([chi, chi[:1], [-1]]).astype(np.int32)
    ids, num = binding.paged_attn_pages_free(dbt, dsl, dref, _i32(rows_))
    st, want, n = pages.free(bt, sl, ref, rows_)
    assert binding.paged_attn_device_status() == st == 0
    assert np.array_equal(ids.cpu().numpy(), want) and num.item() == n
    assert np.array_equal(dref.cpu().numpy(), ref) and np.array_equal(ref, ref0)
    assert np.array_equal(dsl.cpu().numpy(), sl)


def test_refused_forks():
    r = np.random.default_rng(9)
    bt, sl, ref, spare = _pool(r, 60, 12, [33, 20, 64, 5], 4)
    caches = _caches(60, ["q4"])
    s = spare
    par = np.array([0, 12, 1, 3, 2, 0, 0, 1, 0, 5, 1, 0, 3, -1], dtype=np.int32)
    chi = np.array([4, 5, 12, 1, 6, 6, 7, 8, 9, 4, 10, -3, 11, 4], dtype=np.int32)
    #  taken, parent out of range, child out of range, child not empty, full length (no page), child twice,
    #  page taken by an earlier entry, page in use, page past the pool, child of row 5 is empty parent but
    #  4 twice, negative page where one is needed, padding, taken, padding
    new = np.array([s[0], s[1], s[2], s[3], s[4], s[5], s[0], bt[0, 0], 60, s[6], -1, s[7], s[8], s[9]], dtype=np.int32)
    _fork(caches, bt, sl, ref, par, chi, new, status=binding.STATUS_PAGE_OP)
    assert new.tolist() == [s[0]] + [-1] * 11 + [s[8], -1]


def test_a_parent_longer_than_its_row_and_bad_ids():
    r = np.random.default_rng(10)
    bt, sl, ref, spare = _pool(r, 30, 5, [48, 40], 3)
    sl[0] = 49                                   # needs four entries, the row has three
    bt[1, 0], bt[1, 2] = 30, -4                  # ids out of range in a shared and in a copied place
    caches = _caches(30, ["q4"])
    _fork(caches, bt, sl, ref, np.array([0, 1], dtype=np.int32), np.array([2, 3], dtype=np.int32),
          spare[:2].astype(np.int32), status=binding.STATUS_PAGE_OP | binding.STATUS_PAGE_RANGE)


def test_free_reports_bad_state():
    bt = np.array([[0, 1, 2], [2, 7, -1], [3, 4, 5]], dtype=np.int32)
    sl = np.array([48, 30, 80], dtype=np.int32)           # the last: five pages, three entries
    ref = np.array([1, 0, 2, 1, 1, 1, 0], dtype=np.int32)
    dev = [_i32(x) for x in (bt, sl, ref)]
    rows = np.array([0, 1, 2, 3, -1], dtype=np.int32)
    ids, num = binding.paged_attn_pages_free(*dev, _i32(rows))
    st, want, n = pages.free(bt, sl, ref, rows)
    assert binding.paged_attn_device_status() == st == (binding.STATUS_PAGE_OP | binding.STATUS_PAGE_RANGE |
                                                        binding.STATUS_SEQ_LEN)
    assert np.array_equal(ids.cpu().numpy(), want) and num.item() == n
    assert np.array_equal(dev[2].cpu().numpy(), ref) and np.array_equal(dev[1].cpu().numpy(), sl)
    # no rows: the list alone
    ids, num = binding.paged_attn_pages_free(*dev, _i32([]))
    assert num.item() == n


@pytest.mark.parametrize("nb", [1, 31, 33, 257, 5000, 70001])
def test_free_list_of_any_pool(nb):
    r = np.random.default_rng(nb)
    ref = r.integers(0, 3, nb).astype(np.int32)
    ids, num = binding.paged_attn_pages_free(_i32([[0]]), _i32([0]), _i32(ref), _i32([-1]))
    free = np.flatnonzero(ref == 0)
    assert num.item() == len(free)
    assert np.array_equal(ids.cpu().numpy(), np.concatenate([free, np.full(nb - len(free), -1)]))


@pytest.mark.parametrize("nb,frac,rows", [(1, 1.0, 1), (1, 0.0, 1), (33, 0.5, 3), (64, 0.0, 2), (64, 1.0, 2),
                                          (500, 0.1, 7), (500, 0.9, 7), (9000, 0.5, 40)])
def test_compact(nb, frac, rows):
    r = np.random.default_rng(nb)
    used = r.permutation(nb)[:int(round(frac * nb))]
    ref = np.zeros(nb, dtype=np.int32)
    ref[used] = r.integers(1, 5, len(used))
    if nb > 60 and frac < 1:
        ref[np.flatnonzero(ref == 0)[-3:]] = -2
    bt = np.full((rows, 40), -1, dtype=np.int32)
    bt[:] = r.integers(-2, nb + 3, bt.shape)              # used ids, free ids and ids out of range
    caches = _caches(nb, ["q4", "scale", "padded", "kv"], nb)
    host = [_raw(c) for c in caches]
    wide = _i32(np.pad(bt, ((0, 0), (0, 3)), constant_values=77))
    dbt, dref = wide[:, :40], _i32(ref)
    page_map, num = binding.paged_attn_pages_compact(caches, dbt, dref)
    st, want, n = pages.compact(host, bt, ref)
    assert binding.paged_attn_device_status() == st
    assert num.item() == n and np.array_equal(page_map.cpu().numpy(), want)
    assert np.array_equal(dref.cpu().numpy(), ref) and np.array_equal(dbt.cpu().numpy(), bt)
    assert (wide[:, 40:] == 77).all()
    for c, h in zip(caches, host):                        # pages past U keep whatever they held
        assert np.array_equal(_raw(c)[:n], h[:n])
    again, num2 = binding.paged_attn_pages_compact(caches, dbt, dref)
    assert num2.item() == n and np.array_equal(again.cpu().numpy(),
                                               np.where(np.arange(nb) < n, np.arange(nb), -1))


def test_a_chain_in_one_graph_replayed():
    """Fork, free and compact captured together on a side stream and replayed on new state."""
    r = np.random.default_rng(21)
    bt, sl, ref, spare = _pool(r, 80, 10, [100, 37, 16, 250], 20)
    par, chi, new = (np.array(x, dtype=np.int32) for x in ([0, 1, 3], [5, 6, 7], spare[:3]))
    rows = np.array([1, 6], dtype=np.int32)
    caches = _caches(80, ["q4", "scale"], 21)
    dev = [_i32(x) for x in (bt, sl, ref, par, chi, new)]
    drows, ids, num = _i32(rows), _i32(np.zeros(80)), _i32([0])
    pmap, used = _i32(np.zeros(80)), _i32([0])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        binding.paged_attn_pages_fork(caches, *dev)
        binding.paged_attn_pages_free(dev[0], dev[1], dev[2], drows, ids, num)
        binding.paged_attn_pages_compact(caches, dev[0], dev[2], pmap, used)
    for _ in range(2):
        host = [_raw(c) for c in caches]
        graph.replay()
        torch.cuda.synchronize()
        pages.fork(host, bt, sl, ref, par, chi, new)
        _, want, n = pages.free(bt, sl, ref, rows)
        _, wmap, u = pages.compact(host, bt, ref)
        assert np.array_equal(ids.cpu().numpy(), want) and num.item() == n
        assert np.array_equal(pmap.cpu().numpy(), wmap) and used.item() == u
        for d, h in zip(dev, (bt, sl, ref, par, chi, new)):
            assert np.array_equal(d.cpu().numpy(), h)
        for c, h in zip(caches, host):
            assert np.array_equal(_raw(c)[:u], h[:u])
        # the next round forks into the rows freed, from the rows still there
        sl[[5, 7]] = 0
        new[:] = np.flatnonzero(ref == 0)[:3]
        dev[1].copy_(_i32(sl))
        dev[5].copy_(_i32(new))
    binding.paged_attn_device_status()


@pytest.mark.parametrize("nb", [2_200_003, 4_500_000])
def test_pools_past_the_masks_in_shared_memory(nb):
    """Free list and compaction of pools whose use masks do not fit the kernels' shared memory."""
    r = np.random.default_rng(nb)
    ref = (r.random(nb) < 0.7).astype(np.int32) * r.integers(1, 4, nb).astype(np.int32)
    dref = _i32(ref)
    ids, num = binding.paged_attn_pages_free(_i32([[0]]), _i32([0]), dref, _i32([-1]))
    free = np.flatnonzero(ref == 0)
    assert num.item() == len(free)
    assert np.array_equal(ids.cpu().numpy(), np.concatenate([free, np.full(nb - len(free), -1)]))
    cache = torch.arange(nb, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2)
    bt = r.integers(-1, nb, (3, 1000)).astype(np.int32)
    dbt = _i32(bt)
    page_map, used = binding.paged_attn_pages_compact([cache], dbt, dref)
    U = nb - len(free)
    high, holes = np.flatnonzero(ref[U:] > 0) + U, np.flatnonzero(ref[:U] == 0)
    want = np.where(ref > 0, np.arange(nb), -1)
    want[high] = holes
    assert used.item() == U and np.array_equal(page_map.cpu().numpy(), want)
    after = np.zeros(nb, dtype=np.int32)
    after[:U] = ref[:U]
    after[holes] = ref[high]
    assert np.array_equal(dref.cpu().numpy(), after)
    home = np.arange(U)
    home[holes] = high
    assert np.array_equal(cache[:U].cpu().numpy(), np.stack([home, home], 1))
    moved = np.where(bt >= 0, want[np.maximum(bt, 0)], -1)
    assert np.array_equal(dbt.cpu().numpy(), np.where(moved >= 0, moved, bt))
    assert binding.paged_attn_device_status() == 0
