"""paged_attn_decode_shared where the prefix kernel is sure to take part: launch forms
that share every prefix, and prefixes that are worth a part of their own.  The plan's list
of skipped pages (the workspace's first int32 a sequence) shows it."""
import numpy as np
import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from tests.walk_cases import Batch

pytestmark = pytest.mark.gpu

FORMS = {"one after the other": {"disable_pdl": True}, "cut to 40": {"num_ctas": 40}, "side by side": {}}
form = pytest.mark.parametrize("form", list(FORMS))
short_form = pytest.mark.parametrize("form", list(FORMS)[:2])   # side by side, prefixes below 16 pages are not shared


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(b, form, dev=None, groups=None, skip=None):
    """(out, lse); the pages that each sequence left to its group must be `skip`, or some."""
    dev = dev or b.on_gpu()
    out, lse = b.buffers()
    gsl, shared = groups or b.groups
    n = binding.paged_attn_shared_workspace_size(
        b.q.shape[0], len(b.lens), b.hq, b.hkv, b.d, binding.PA_FP8_E4M3 if b.kv == "fp8" else binding.PA_BF16, b.runs,
        b.options(**FORMS[form]))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    binding.paged_attn_decode_shared(*dev, b.runs, _i32(gsl), _i32(shared), b.scale, b.ks, b.vs, out=out, lse=lse,
                                     options=b.options(workspace=ws.data_ptr(), workspace_bytes=n, **FORMS[form]))
    torch.cuda.synchronize()
    took = ws[:4 * len(b.lens)].view(torch.int32).cpu().numpy()
    assert (took == skip).all() if skip is not None else took.any(), took
    return out, lse


def _layouts(x):
    """The cache in rows of its heads, with room behind each head, and head by head."""
    nb, _, h, d = x.shape
    wide = torch.zeros(nb, 17, h + 1, d + 16, dtype=x.dtype, device="cuda")
    by_head = torch.zeros(nb, h, 16, d, dtype=x.dtype, device="cuda")
    yield x
    for y in (wide[:, :16, :h, :d], by_head.transpose(1, 2)):
        y.copy_(x)
        yield y


@form
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_every_layout_of_keys_beside_every_one_of_values(kv, d, form):
    # side by side: 40 x 68 pages x 3 heads x 59 ns at least, above the 304 us that are left to the sequences
    b = Batch([1100 + 9 * i for i in range(40)], hq=6, hkv=3, d=d, kv=kv, groups=([0, 40], [1090]))
    dev = b.on_gpu()
    first = None
    for k in _layouts(dev[1]):
        for v in _layouts(dev[2]):
            got = _run(b, form, [dev[0], k, v] + dev[3:], skip=1090 // 16)
            if first is None:
                first = got
                b.check(*got)
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@form
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_replays_over_new_lists(kv, form):
    """A captured call whose lists, lengths, tables and queries change between its replays: every kernel of it works
    on this replay's plan.  The word that says that the plan is there (behind the skipped pages) is taken back."""
    lens = np.concatenate([1200 + 5 * np.arange(60), [40] * 4])
    batches = [Batch(lens, hq=16, hkv=4, d=64, kv=kv, groups=g, seed=7)
               for g in (([0, 30, 60], [1190, 1000]), ([10, 50, 60], [1195, 160]), ([0, 60, 64], [700, 0]))]
    assert all((x.lens == lens).all() and x.bt.shape == batches[0].bt.shape for x in batches)
    pages = max(x.k.shape[0] for x in batches)
    dev = batches[0].on_gpu()
    for x in (1, 2):
        dev[x] = torch.zeros(pages, *dev[x].shape[1:], dtype=dev[x].dtype, device="cuda")
    lists = [_i32([0, 0, 0]), _i32([0, 0])]
    out, lse = batches[0].buffers()
    code = binding.PA_FP8_E4M3 if kv == "fp8" else binding.PA_BF16
    n = binding.paged_attn_shared_workspace_size(64, 64, 16, 4, 64, code, 1, batches[0].options(**FORMS[form]))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    call = binding.prepare_decode_shared(*dev, 1, *lists, batches[0].scale, batches[0].ks, batches[0].vs, out=out, lse=lse,
                                         options=batches[0].options(workspace=ws.data_ptr(), workspace_bytes=n, **FORMS[form]))
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    word = ws[256:264].view(torch.int64)
    for again in range(3):
        for b in batches:
            new = b.on_gpu() + [_i32(b.groups[0]), _i32(b.groups[1])]
            for x, y in zip(dev + lists, new):
                if y is not None:
                    x[:y.shape[0]].copy_(y)
            out.fill_(7.0)
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            assert int(word) == 0 and ws[:256].view(torch.int32).any()
            if again == 0:
                b.check(out, lse)
                b.got = out.clone(), lse.clone()
            assert torch.equal(out, b.got[0]) and torch.equal(lse, b.got[1])


@form
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_scales(kv, d, scale, form):
    b = Batch(1040 + np.arange(40), hq=16, hkv=4, d=d, kv=kv, groups=([0, 40], [1040]), scale=scale)
    b.check(*_run(b, form, skip=64))                            # the newest token of the shortest is page 65's


@form
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_growing_maximum(kv, d, form):
    """Keys whose scores rise block by block: O in tensor memory is rescaled again and again."""
    b = Batch([1284] * 40, hq=8, hkv=2, d=d, kv=kv, groups=([0, 40], [1280]), scale=1.0)
    for j in range(1280):
        page, f = b.bt[0, j // 16], 0.02 + 4.0 * (j // 64) / 20
        if kv == "bf16":
            b.k[page, j % 16] *= f
        else:
            x = b.k[page, j % 16].view(torch.float8_e4m3fn).float() * f
            b.k[page, j % 16] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    b.check(*_run(b, form, skip=80))


@form
@pytest.mark.parametrize("what", ["key", "value", "query", "infinite key"])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_nan_and_infinity_in_a_shared_page(kv, d, what, form):
    if kv == "fp8" and what == "infinite key":
        pytest.skip("the codes have no infinity")
    b = Batch(1000 + np.arange(40), hq=16, hkv=4, d=d, kv=kv, groups=([0, 40], [992]))
    nan = 0x7F if kv == "fp8" else float("nan")
    if what == "key":
        b.k[b.bt[0, 20], 3, 1, 5] = nan
    elif what == "value":
        b.v[b.bt[0, 33], 15, 2, 7] = nan
    elif what == "query":
        b.q[7, 9, 2] = float("nan")
    else:
        b.k[b.bt[0, 20], 3, 1, 5] = float("inf")
    out, lse = _run(b, form, skip=62)
    # (over fp8 caches a query value without a finite f16 sets bit 4, as in every decode call)
    b.check(out, lse, status=binding.STATUS_F16_RANGE if kv == "fp8" and what == "query" else 0)
    gone = torch.isnan(out).any(-1)
    rows = {"key": 40 * 4, "value": 40 * 4, "query": 1, "infinite key": int((b.q[:, 4:8, 5] > 0).sum())}
    assert int(gone.sum()) == rows[what]


def _kinds(n, sinks, **kw):
    """n times over: runs, sequences of no group, a group of one, shared lengths of zero, past the tables' and short of a
    page."""
    qlens = [1, 3] + [2, 1] * n + [1, 3, 3] * n + [2] + [1, 1] * n + [2, 3] * n + [1] * n + [1]
    lens = [300, 290] + [610, 580] * n + [700, 710, 705] * n + [64] + [333, 334] * n + [40, 90] * n + [2000] * n + [7]
    at = np.cumsum([2, 2 * n, 3 * n, 1, 2 * n, 2 * n, n]).tolist()
    return Batch(lens, qlens, hq=12, hkv=3, groups=([2] + at, [999, 570, 690, 40, 300, 0, 9999]), sinks=sinks, **kw)


@form
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_groups_of_every_kind(kv, d, sinks, form):
    b = _kinds(12, sinks, kv=kv, d=d, extra=8)
    b.check(*_run(b, form))


@form
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_padded_batch_and_empty_rows(kv, sinks, form):
    """Members without query tokens or without a context take no part; the group's pages are those of the first that
    does."""
    lens = [0, 900, 890, 0] + [895 + i for i in range(40)] + [2, 899]
    qlens = [1, 2, 0, 0] + [1 + i % 3 for i in range(40)] + [4, 0]
    b = Batch(lens, qlens, hq=8, hkv=2, kv=kv, groups=([0, 46], [880]), sinks=sinks, pad_rows=5)
    b.bt[44, 0] = b.bt[1, 0]
    skip = [0, 55, 0, 0] + [55] * 40 + [0, 0]
    b.check(*_run(b, form, skip=skip), status=binding.STATUS_SEQ_LEN)


@form
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_shared_length_past_a_member_is_cut(kv, form):
    b = Batch([900 + i for i in range(20)] + [400] + [900 + i for i in range(20)], hq=16, hkv=4, kv=kv,
              groups=([0, 41], [896]))
    b.check(*_run(b, form, skip=24))                            # whole pages before the 400th token's


@short_form
def test_short_prefixes_are_cut_and_shared(form):
    b = Batch([500, 160, 500, 490], hq=8, hkv=2, d=64, groups=([0, 4], [480]))
    b.check(*_run(b, form, skip=9))
    b = Batch([160, 160], hq=8, hkv=2, d=64, groups=([0, 2], [160]))     # the newest token's page too
    b.check(*_run(b, form, skip=9))
    b = Batch([17, 33], hq=1, hkv=1, d=128, groups=([0, 2], [16]))
    b.check(*_run(b, form, skip=1))


@form
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("fp8", 64)])
def test_slots_past_the_end_and_free_pages_hold_nan(kv, d, form):
    lens = [801 + 7 * i for i in range(40)]
    b = Batch(lens, hq=16, hkv=4, d=d, kv=kv, groups=([0, 40], [800]))
    nan = float("nan") if kv == "bf16" else 0x7F
    for i, L in enumerate(lens):
        for j in range(L, -(-L // 16) * 16):
            b.k[b.bt[i, j // 16], j % 16] = b.v[b.bt[i, j // 16], j % 16] = nan
    free = sorted(set(range(b.k.shape[0])) - set(b.bt[b.bt >= 0].tolist()))
    b.k[free] = b.v[free] = nan
    b.check(*_run(b, form, skip=50))


@form
@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_bad_page_id_of_a_shared_page(kv, d, bad, form):
    """Reported; the other group's rows are as without it."""
    b = Batch(1000 + np.arange(60), hq=16, hkv=4, d=d, kv=kv, groups=([0, 30, 60], [992, 980]))
    want = _run(b, form)
    assert binding.paged_attn_device_status() == 0
    b.bt[0, 20] = bad
    got = _run(b, form)
    assert binding.paged_attn_device_status(clear=True) == binding.STATUS_PAGE_RANGE
    assert torch.equal(got[0][30:], want[0][30:]) and torch.equal(got[1][30:], want[1][30:])


def test_library_workspace_and_capture():
    import ctypes
    b = Batch([1000 + i for i in range(60)], hq=8, hkv=2, groups=([0, 60], [1000]))
    _run(b, "side by side", skip=62)
    lib = binding.load()
    dev = b.on_gpu() + [_i32([0, 60]), _i32([1000])]
    binding.paged_attn_release()
    binding.paged_attn_shared_reserve(60, 60, 8, 2, 128)
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


@form
def test_a_serving_step(form):
    """A prompt written with positions and forked to a batch, a token for each, decode over the shared pages."""
    r = np.random.default_rng(1)
    hq, hkv, d, L, n = 16, 4, 64, 1333, 47
    nb = 84 + 2 * n
    ang = np.arange(1400)[:, None] * 10000.0 ** (-2.0 * np.arange(d // 2) / d)[None]
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    kc, vc = (torch.zeros(nb, 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.full((n + 1, 90), -1, dtype=torch.int32, device="cuda")
    order = torch.from_numpy(r.permutation(nb).astype(np.int32)).cuda()
    bt[0, :84] = order[:84]
    sl = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    sl[0] = L
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    ref[order[:84].long()] = 1
    gen = torch.Generator(device="cuda").manual_seed(2)
    mk = lambda t, h: torch.randn(t, h, d, device="cuda", generator=gen).to(torch.bfloat16)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    slots = (bt[0].long()[pos.long() // 16] * 16 + pos % 16).int()
    binding.paged_attn_rope_cache_write(mk(L, hq), mk(L, hkv), mk(L, hkv), pos, table, slots, kc, vc)
    binding.paged_attn_pages_fork([kc, vc], bt, sl, ref, _i32([0] * n), _i32(list(range(1, n + 1))),
                                  order[84:84 + n].contiguous())
    pos = _i32([L] * (n + 1))
    slots = (bt[:, L // 16].long() * 16 + L % 16).int()
    q = binding.paged_attn_rope_cache_write(mk(n + 1, hq), mk(n + 1, hkv), mk(n + 1, hkv), pos, table, slots, kc, vc)
    sl += 1
    b = Batch([L + 1] * (n + 1), hq=hq, hkv=hkv, d=d, groups=([0, n + 1], [L]))
    b.on_gpu()
    got = _run(b, form, [q, kc, vc, bt, sl, None], skip=L // 16)
    assert binding.paged_attn_device_status() == 0
    b.q, b.k, b.v, b.bt = q.cpu(), kc.cpu(), vc.cpu(), bt.cpu().numpy()
    b.check(*got)
