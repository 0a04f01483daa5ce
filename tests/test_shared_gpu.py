"""paged_attn_decode_shared against the float64 oracle (of ordinary decode on the same
block tables)."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(b, groups=None, **kw):
    dev = b.on_gpu()
    out, lse = b.buffers()
    gsl, shared = groups or b.groups
    binding.paged_attn_decode_shared(*dev, b.runs, _i32(gsl), _i32(shared), b.scale, b.ks, b.vs, out=out, lse=lse,
                                     options=b.options(**kw))
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,shared,hq,hkv", [(2, 16, 1, 1), (4, 100, 8, 2), (16, 128, 8, 1), (17, 144, 8, 1),
                                             (33, 400, 8, 2), (40, 1000, 8, 1), (7, 2100, 5, 5), (64, 530, 32, 8)])
def test_one_group(n, shared, hq, hkv, d, kv):
    r = np.random.default_rng(n)
    lens = shared + r.integers(1, 90, n)
    b = Batch(lens, hq=hq, hkv=hkv, d=d, kv=kv, groups=([0, n], [shared]), seed=n)
    b.check(*_run(b))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_groups_of_every_kind(kv):
    """Runs, sequences of no group, groups of one, shared lengths of zero, past the tables' and short of a page."""
    qlens = [1, 3, 2, 1, 1, 3, 3, 2, 1, 1, 2, 3, 1, 1]
    lens = [300, 290, 410, 50, 700, 710, 705, 64, 33, 34, 40, 90, 2000, 7]
    b = Batch(lens, qlens, hq=12, hkv=3, d=128, kv=kv, groups=([2, 2, 4, 7, 8, 10, 12, 13], [500, 16, 690, 40, 15, 0, 999]),
              sinks=True)
    b.check(*_run(b))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctas", [0, 1, 3, 40])
def test_many_rows_and_pieces(ctas, kv):
    """Several tile pairs a head, the last with one tile or two; pieces cut by CTAs."""
    for n, hq, hkv in ((70, 8, 1), (100, 8, 2), (129, 4, 1)):
        r = np.random.default_rng(n)
        b = Batch(1500 + r.integers(1, 40, n), hq=hq, hkv=hkv, d=64, kv=kv, groups=([0, n], [1500]), seed=n)
        b.check(*_run(b, num_ctas=ctas))


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_long_prefix_few_rows(kv, d):
    b = Batch([30050, 30040, 30033], hq=8, hkv=2, d=d, kv=kv, groups=([0, 3], [30032]))
    b.check(*_run(b))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_scales(scale, kv):
    b = Batch([300, 301, 290, 333], hq=8, hkv=2, d=64, kv=kv, groups=([0, 4], [280]), scale=scale)
    b.check(*_run(b))


def test_growing_maximum():
    """Keys whose scores rise block by block: O is rescaled again and again."""
    b = Batch([900] * 20, hq=8, hkv=2, d=64, groups=([0, 20], [896]), scale=1.0)
    for j in range(900):
        b.k[b.bt[0, j // 16], j % 16] *= 0.02 + 4.0 * (j // 64) / 14
    b.check(*_run(b))


def test_shared_length_past_a_member_is_cut():
    lens = [500, 160, 500, 490]
    b = Batch(lens, hq=8, hkv=2, d=64, groups=([0, 4], [480]))
    assert (b.bt[1, :10] == b.bt[0, :10]).all()
    b.check(*_run(b))
    b = Batch([160, 160], hq=8, hkv=2, d=64, groups=([0, 2], [160]))     # the newest token's page too
    b.check(*_run(b))


@pytest.mark.parametrize("sinks", [False, True])
def test_padded_batch_and_empty_rows(sinks):
    b = Batch([0, 300, 290, 0, 305, 2, 299], [1, 2, 0, 0, 3, 4, 1], hq=8, hkv=2, d=64, groups=([0, 7], [288]), sinks=sinks,
              pad_rows=5)
    b.bt[5, 0] = b.bt[1, 0]
    b.check(*_run(b), status=binding.STATUS_SEQ_LEN)


def test_padding_alone_sets_no_status():
    b = Batch([290, 0, 300, 0], [2, 0, 1, 0], hq=8, hkv=2, d=64, groups=([0, 4], [280]), pad_rows=3)
    b.check(*_run(b))


def test_no_groups():
    b = Batch([100, 40], hq=8, hkv=2)
    b.check(*_run(b, ([0], [])))
    dev = b.on_gpu()
    out, lse = binding.paged_attn_decode_shared(*dev, 1, _i32([0]), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                                b.scale)
    assert (out - _run(b, ([0], []))[0]).abs().max() == 0


@pytest.mark.parametrize("groups", [([0, 5, 3, 4], [96, 96, 96]), ([-1, 4], [96]), ([0, 9], [96]), ([3, 1], [96])])
def test_bad_groups_share_nothing(groups):
    b = Batch([100, 110, 120, 130], hq=8, hkv=2, d=64, groups=([0, 4], [96]))
    b.check(*_run(b, groups), status=binding.STATUS_QUERY_LEN)


def test_nan_is_not_lost_and_stays_in_its_head():
    b = Batch([600] * 6, hq=8, hkv=2, d=64, groups=([0, 6], [592]))
    b.k[b.bt[0, 20], 3, 0] = float("nan")
    out, lse = _run(b)
    assert torch.isnan(out[:, :4]).all() and torch.isnan(lse[:, :4]).all() and torch.isfinite(out[:, 4:]).all()
    b = Batch([600] * 6, hq=8, hkv=2, d=64, groups=([0, 6], [592]))
    b.q[2, 1] = float("nan")
    out, lse = _run(b)
    assert torch.isnan(out[2, 1]).all() and torch.isnan(lse[2, 1]) and int(torch.isnan(out).any(-1).sum()) == 1


def test_slots_past_the_end_and_free_pages_hold_nan():
    lens = [205, 210, 230, 199]
    b = Batch(lens, hq=8, hkv=2, d=64, groups=([0, 4], [192]))
    for i, L in enumerate(lens):
        for j in range(L, -(-L // 16) * 16):
            b.k[b.bt[i, j // 16], j % 16] = b.v[b.bt[i, j // 16], j % 16] = float("nan")
    free = sorted(set(range(b.k.shape[0])) - set(b.bt[b.bt >= 0].tolist()))
    b.k[free] = b.v[free] = float("nan")
    b.check(*_run(b))


def test_bad_page_id_is_reported():
    b = Batch([200, 210, 220], hq=4, hkv=2, groups=([0, 3], [192]))
    b.bt[0, 2] = b.k.shape[0]
    _run(b)
    assert binding.paged_attn_device_status() & binding.STATUS_PAGE_RANGE


@pytest.mark.parametrize("kw", [dict(num_ctas=2), dict(min_pages_per_cta=1), dict(heads_per_cta=1), dict(disable_pdl=True),
                                dict(page_pairing=1), dict(num_ctas=500)])
def test_launch_forms(kw):
    b = Batch([700 + 3 * i for i in range(30)], [1 + i % 3 for i in range(30)], hq=8, hkv=2, groups=([0, 12, 30], [690, 720]))
    b.check(*_run(b, **kw))


def test_graphs_streams_and_prepared_calls():
    b = Batch([1000 + 7 * i for i in range(24)], hq=8, hkv=2, groups=([0, 10, 24], [992, 500]))
    dev = b.on_gpu()
    lists = [(_i32([0, 10, 24]), _i32([992, 500])), (_i32([10, 24]), _i32([480]))]
    calls = [binding.prepare_decode_shared(*dev, 1, *x, b.scale) for x in lists]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls[0]()
    calls[1]()
    torch.cuda.synchronize()
    for c in calls:
        b.check(c.out, c.lse)
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for c in calls:
        c.out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
    torch.cuda.synchronize()
    for c in calls:
        b.check(c.out, c.lse)


def test_library_workspace_and_capture():
    b = Batch([400 + i for i in range(16)], hq=8, hkv=2, groups=([0, 16], [400]))
    import ctypes
    lib = binding.load()
    dev = b.on_gpu() + [_i32([0, 16]), _i32([400])]
    binding.paged_attn_release()
    binding.paged_attn_shared_reserve(16, 16, 8, 2, 128)
    out, lse = b.buffers()
    r = [ctypes.byref(binding.tensor_desc(t)) for t in dev + [out, lse]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = lib.paged_attn_decode_shared(*r[:6], 1, r[6], r[7], b.scale, 1.0, 1.0, r[8], r[9], None,
                                          torch.cuda.current_stream().cuda_stream)
    assert st == binding.PA_OK, binding.paged_attn_last_error_message()
    g.replay()
    torch.cuda.synchronize()
    b.check(out, lse)


def test_a_serving_step():
    """Positions and cache write, fork, decode over the shared pages, decode over a window: one after another."""
    from oracle import rope
    r = np.random.default_rng(0)
    hq, hkv, d, L, n = 8, 2, 64, 333, 5
    nb = 60
    ang = np.arange(400)[:, None] * 10000.0 ** (-2.0 * np.arange(d // 2) / d)[None]
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    kc, vc = (torch.zeros(nb, 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.full((n + 1, 24), -1, dtype=torch.int32, device="cuda")
    order = torch.from_numpy(r.permutation(nb).astype(np.int32)).cuda()
    bt[0, :21] = order[:21]
    sl = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    ref[order[:21].long()] = 1
    # a prompt
    mk = lambda t, h: torch.randn(t, h, d, device="cuda").to(torch.bfloat16)
    q, k, v = mk(L, hq), mk(L, hkv), mk(L, hkv)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    slots = (bt[0].long()[pos.long() // 16] * 16 + pos % 16).int()
    binding.paged_attn_rope_cache_write(q, k, v, pos, table, slots, kc, vc)
    sl[0] = L
    # branched
    children = _i32(list(range(1, n + 1)))
    new = order[21:21 + n].contiguous()
    binding.paged_attn_pages_fork([kc, vc], bt, sl, ref, _i32([0] * n), children, new)
    assert (sl == L).all()
    # a new token for each sequence
    q, k, v = mk(n + 1, hq), mk(n + 1, hkv), mk(n + 1, hkv)
    pos = _i32([L] * (n + 1))
    slots = (bt[:, L // 16].long() * 16 + L % 16).int()
    qr = binding.paged_attn_rope_cache_write(q, k, v, pos, table, slots, kc, vc)
    sl += 1
    out, lse = binding.paged_attn_decode_shared(qr, kc, vc, bt, sl, None, 1, _i32([0, n + 1]), _i32([L]))
    ref_out, ref_lse = binding.paged_attn_decode(qr, kc, vc, bt, sl)
    win, _ = binding.paged_attn_decode_window(qr, kc, vc, bt, sl, None, 1, 100, 4)
    torch.cuda.synchronize()
    assert binding.paged_attn_device_status() == 0
    want = rope.rotate(q.float().cpu().numpy(), np.full((1, n + 1), L), table.cpu().numpy(), None, False, np.float32)
    assert (rope.bf16_bits(want) == qr.view(torch.int16).cpu().numpy().view(np.uint16)).all()
    b = Batch([L + 1] * (n + 1), hq=hq, hkv=hkv, d=d)
    b.q, b.k, b.v, b.bt = qr.cpu(), kc.cpu(), vc.cpu(), bt.cpu().numpy()
    b.check(out, lse)
    b.check(ref_out, ref_lse)
    assert np.abs(win.double().cpu().numpy() - b.want(100, 4)[0]).max() < 2.0 ** -6


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_heads_that_are_not_contiguous(kv, d):
    b = Batch([700 + 9 * i for i in range(9)], hq=6, hkv=3, d=d, kv=kv, groups=([0, 9], [690]))
    dev = b.on_gpu()
    for x in (1, 2):
        wide = torch.zeros(dev[x].shape[0], 17, 4, d + 16, dtype=dev[x].dtype, device="cuda")
        wide[:, :16, :3, :d] = dev[x]
        dev[x] = wide[:, :16, :3, :d]
    out, lse = b.buffers()
    binding.paged_attn_decode_shared(*dev, 1, _i32([0, 9]), _i32([690]), b.scale, b.ks, b.vs, out=out, lse=lse)
    torch.cuda.synchronize()
    b.check(out, lse)


@pytest.mark.parametrize("kv,d", [("fp8", 128), ("bf16", 128), ("fp8", 64), ("bf16", 64)])
@pytest.mark.parametrize("ctas", [1, 5, 152])
def test_many_pieces_a_cta(kv, d, ctas):
    """Pieces of every form one after another in a CTA: single tiles, pairs, odd blocks, short last blocks."""
    r = np.random.default_rng(d + ctas)
    sizes, shared = [2, 3, 34, 20, 9, 2, 40, 5], [130, 16, 700, 1040, 2000, 129 * 16, 64, 1500]
    lens = np.concatenate([s + r.integers(1, 30, n) for n, s in zip(sizes, shared)])
    b = Batch(lens, hq=16, hkv=2, d=d, kv=kv, groups=(np.concatenate([[0], np.cumsum(sizes)]).tolist(), shared), seed=1)
    b.check(*_run(b, num_ctas=ctas))


_FORMS = {"one after the other": {"disable_pdl": True}, "side by side": {}, "cut to 40": {"num_ctas": 40}}


@pytest.mark.parametrize("form", list(_FORMS))
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,shared,hq,hkv", [(2, 16, 1, 1), (3, 130, 16, 2), (16, 128, 8, 1), (17, 255, 8, 1),
                                             (33, 272, 8, 2), (40, 1000, 8, 1), (7, 2100, 5, 5), (90, 650, 16, 4)])
def test_every_form_of_one_group(n, shared, hq, hkv, d, kv, form):
    """Short prefixes are left to the sequences where both parts run side by side, and shared elsewhere."""
    r = np.random.default_rng(n + shared)
    b = Batch(shared + r.integers(1, 90, n), hq=hq, hkv=hkv, d=d, kv=kv, groups=([0, n], [shared]), seed=n)
    b.check(*_run(b, **_FORMS[form]))


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("fp8", 128)])
def test_short_and_long_prefixes_side_by_side(kv, d):
    """Groups on both sides of the shortest shared prefix, and sequences of no group."""
    sizes, shared = [30, 20, 40, 10], [255, 256, 500, 1600]
    r = np.random.default_rng(d)
    lens = np.concatenate([s + r.integers(1, 200, n) for n, s in zip(sizes, shared)] + [r.integers(1, 900, 20)])
    b = Batch(lens, hq=16, hkv=4, d=d, kv=kv, groups=(np.concatenate([[0], np.cumsum(sizes)]).tolist(), shared), seed=2)
    b.check(*_run(b))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_the_same_rows_every_time(kv):
    """The two parts run beside each other: no call's result depends on their timing."""
    r = np.random.default_rng(5)
    lens = 1300 + r.integers(1, 300, 60)
    b = Batch(lens, hq=32, hkv=4, d=128, kv=kv, groups=([0, 25, 60], [1290, 1000]), seed=3)
    out, lse = _run(b)
    b.check(out, lse)
    for _ in range(20):
        o, l = _run(b)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_as_many_sequences_as_a_call_takes():
    r = np.random.default_rng(8)
    sizes = r.integers(1, 60, 400)
    sizes = sizes[np.cumsum(sizes) <= 8000]
    shared = r.choice([0, 17, 250, 256, 300, 700], len(sizes))
    lens = np.concatenate([s + r.integers(1, 20, n) for n, s in zip(sizes, shared)])
    lens = np.concatenate([lens, r.integers(1, 40, 8192 - len(lens))])
    at = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    b = Batch(lens, hq=2, hkv=1, d=64, kv="bf16", groups=(at, shared.tolist()), seed=4)
    b.check(*_run(b))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_wait_limit_alone_changes_nothing(kv):
    b = Batch(900 + np.arange(50), hq=16, hkv=2, d=128, kv=kv, groups=([0, 50], [890]), seed=6)
    out, lse = _run(b)
    o, l = _run(b, wait_limit_us=50000)
    b.check(o, l)
    assert torch.equal(o, out) and torch.equal(l, lse)
