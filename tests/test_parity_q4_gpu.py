"""paged_attn_decode_q4 against the float64 oracle on the same codes and scales."""
import numpy as np
import pytest
import torch

from oracle import cache_q4
from paged_kv_decode_06_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    binding.paged_attn_device_status(clear=True)
    yield


class Case:
    """A batch over a 4-bit cache: seeded codes and scales, permuted pages."""

    def __init__(self, lens, qlens=None, hq=8, hkv=2, d=128, seed=0, k_scale=0.02, v_scale=0.03, window=0, sinks=False,
                 scale=None, extra_pages=3, pad_rows=0, q_gain=1.0):
        r = np.random.default_rng(seed)
        self.lens = np.array(lens, dtype=np.int32)
        self.qlens = np.ones(len(lens), dtype=np.int64) if qlens is None else np.array(qlens)
        self.qsl = None if qlens is None else np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.runs = 1 if qlens is None else max(1, int(self.qlens.max()))
        self.hq, self.hkv, self.d, self.window = hq, hkv, d, window
        self.k_scale, self.v_scale = k_scale, v_scale
        self.scale = d ** -0.5 if scale is None else scale
        n = -(-np.maximum(self.lens, 0) // 16)
        nb = int(n.sum()) + extra_pages
        order = r.permutation(nb)
        self.bt = np.full((len(lens), max(1, int(n.max()))), -1, dtype=np.int32)
        at = 0
        for i, k in enumerate(n):
            self.bt[i, :k] = order[at:at + k]
            at += k
        self.codes = [r.integers(0, 256, (nb, 16, hkv, d // 2)).astype(np.uint8) for _ in range(2)]
        # group scales 2^-3 .. 2^5 (codes 0x20 .. 0x5F), as rows of varying size have
        self.scales = [r.integers(0x20, 0x60, (nb, hkv, 16, d // 16)).astype(np.uint8) for _ in range(2)]
        t = int(self.qlens.sum()) + pad_rows
        q = r.standard_normal((t, hq, d)) * q_gain
        self.q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
        self.sinks = r.standard_normal(hq).astype(np.float32) if sinks else None

    def on_gpu(self):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.dev = [self.q.cuda(), c(self.codes[0]), c(self.codes[1]), c(self.scales[0]), c(self.scales[1]), c(self.bt),
                    c(self.lens), None if self.qsl is None else c(self.qsl)]
        self.dsinks = None if self.sinks is None else c(self.sinks)
        return self.dev

    def options(self, **kw):
        return binding.make_options(sliding_window=self.window, sinks=getattr(self, "dsinks", None), **kw)

    def run(self, **kw):
        dev = self.on_gpu()
        out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        binding.paged_attn_decode_q4(*dev, self.runs, self.scale, self.k_scale, self.v_scale, out=out, lse=lse,
                                     options=self.options(**kw))
        torch.cuda.synchronize()
        return out, lse

    def want(self):
        return cache_q4.decode(self.q.double().numpy(), self.codes, self.scales, self.bt, self.lens, self.qsl,
                               self.scale, self.k_scale, self.v_scale, self.window, self.sinks)

    def check(self, out, lse, status=0):
        """Every row against the oracle, within the sum of the roundings on the way:
        bf16 output 2^-8; f16 weights 2^-11 (and 2^-25 of the largest for the smallest ones, of N keys);
        fp32 sums of N terms N 2^-24 twice (weights, outputs); exponentials 2^-21;
        scores: fp32 sums of D products, (D + 4) 2^-24 of sum |q k|, query elements in f16 2^-25 of the
        row's largest (elements below its 2^-14), a relative error of the weights of the same size."""
        assert binding.paged_attn_device_status() == status
        wo, wl = self.want()
        go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        k, v = [cache_q4.dequantise_rows(self.codes[x], self.scales[x].transpose(0, 2, 1, 3),
                                         (self.k_scale, self.v_scale)[x]) for x in range(2)]
        kmax, vmax = np.nanmax(np.abs(k)), np.nanmax(np.abs(v))
        n = max(1, int(self.lens.max()))
        aq = np.abs(self.q.double().numpy())
        ds = abs(self.scale) * kmax * (aq.sum(-1) * (self.d + 4) * 2.0 ** -24 + self.d * 2 * aq.max(-1) * 2.0 ** -25)
        ds = ds + 2.0 ** -20 * 1.5                         # log2 e and the product with the row's factor
        w = 2 * (2.0 ** -11 + n * 2.0 ** -25 + n * 2.0 ** -23 + 2.0 ** -21 + ds)
        rows = ~np.isnan(wl) | np.isneginf(wl)
        fill = np.isnan(wo).all(-1) & np.isnan(wl) & (np.arange(len(wl)) >= (self.qlens.sum()))[:, None]
        assert (go[fill] == 7).all() and (gl[fill] == 7).all()      # rows of no sequence stay as they were
        live = ~fill
        assert np.array_equal(np.isnan(wo[live]), np.isnan(go[live]))
        assert np.array_equal(np.isnan(wl[live]), np.isnan(gl[live]))
        with np.errstate(invalid="ignore"):
            err = np.abs(go - wo)
            tol = 2.0 ** -8 * np.abs(wo) * (1 + 2.0 ** -7) + (w * vmax)[..., None]
            assert (np.isnan(err) | (err <= tol))[live].all(), np.nanmax((err / tol)[live])
            inf = np.isneginf(wl)
            assert np.array_equal(inf[live], np.isneginf(gl)[live])
            el = np.abs(gl - wl)
            tl = ds + n * 2.0 ** -23 + 2.0 ** -20 + np.abs(wl) * 2.0 ** -21
            assert (np.isnan(el) | inf | (el <= tl))[live].all(), np.nanmax(el[live & rows])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [31, 32, 33, 100], [1, 2, 400]])
def test_page_boundaries(d, lens):
    c = Case(lens, d=d, seed=len(lens) + d)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (7, 1, 128), (8, 1, 64), (6, 3, 128), (40, 5, 64), (20, 10, 128),
                                      (16, 16, 64), (9, 9, 128), (22, 11, 64), (14, 7, 128), (12, 12, 128),
                                      (16, 1, 128), (64, 1, 64), (32, 2, 128), (64, 2, 128), (36, 4, 64)])
def test_head_layouts(hq, hkv, d):
    c = Case([70, 5, 129], hq=hq, hkv=hkv, d=d, seed=hq + hkv)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,qlens", [(8, 2, [1, 2, 3]), (8, 8, [7, 1, 4]), (64, 8, [4, 1, 3]), (16, 1, [1, 4, 2]),
                                          (1, 1, [64, 1, 30]), (24, 3, [2, 5, 8]), (20, 4, [12, 3, 1]), (6, 2, [1, 1, 1])])
@pytest.mark.parametrize("d", [64, 128])
def test_query_runs(hq, hkv, qlens, d):
    c = Case([64, 77, 210], qlens, hq=hq, hkv=hkv, d=d, seed=sum(qlens))
    c.check(*c.run())


@pytest.mark.parametrize("window", [1, 5, 16, 17, 50, 1000])
@pytest.mark.parametrize("qlens", [None, [3, 1, 4]])
def test_windows_and_sinks(window, qlens):
    c = Case([64, 7, 210], qlens, hq=8, hkv=2, d=64 if qlens else 128, window=window, sinks=window % 2 == 0, seed=window)
    c.check(*c.run())


@pytest.mark.parametrize("ctas", [1, 2, 7, 33, 200, 700])
@pytest.mark.parametrize("hq,hkv,d,qlens", [(8, 2, 128, None), (8, 1, 64, None), (32, 4, 64, [2, 1, 2, 1]),
                                            (48, 3, 128, [1, 3, 2, 1])])
def test_forced_splits(ctas, hq, hkv, d, qlens):
    c = Case([300, 17, 1, 650], qlens, hq=hq, hkv=hkv, d=d, sinks=ctas % 2 == 1, seed=ctas)
    # the third sequence's run of 2 is longer than its one cached token
    c.check(*c.run(num_ctas=ctas, min_pages_per_cta=1), status=binding.STATUS_SEQ_LEN if qlens else 0)


@pytest.mark.parametrize("heads", [1, 2, 4, 8])
def test_heads_per_cta(heads):
    c = Case([90, 300], hq=32, hkv=8, seed=heads)
    c.check(*c.run(heads_per_cta=heads))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("ks,vs", [(0.02, 0.03), (-0.5, 1.0)])
def test_softmax_scales(scale, ks, vs):
    c = Case([40, 130], scale=scale, k_scale=ks, v_scale=vs, seed=9)
    c.check(*c.run())


@pytest.mark.parametrize("gain", [1e-20, 1e-5, 1e4, 1e20])
def test_query_rows_of_any_size(gain):
    c = Case([40, 130], [2, 1], q_gain=gain, k_scale=0.02 / gain, seed=10)
    c.check(*c.run())


def test_long_scores_move_the_maximum():
    """Scores that grow along the sequence by more than the threshold, in both directions."""
    for seed in range(2):
        c = Case([500, 333], hq=8, hkv=2, d=64, seed=seed, scale=2.0)
        n = c.bt.shape[1]
        for i in range(2):
            for j, p in enumerate(c.bt[i]):
                if p >= 0:
                    c.scales[0][p] = 0x20 + (j if seed else n - j)
        c.check(*c.run())


def test_padded_batch():
    """Sequences without query tokens, without keys, and rows of no sequence."""
    c = Case([40, 0, 33, 0, 100, 20], [2, 0, 1, 1, 0, 3], hq=8, hkv=2, sinks=True, pad_rows=5, seed=11)
    c.check(*c.run(), status=binding.STATUS_SEQ_LEN)
    c = Case([40, 0, 2], [1, 2, 4], hq=8, hkv=2, seed=12)           # more query tokens than keys
    c.check(*c.run(num_ctas=3, min_pages_per_cta=1), status=binding.STATUS_SEQ_LEN)
    c = Case([0, 0], [0, 0], pad_rows=2, seed=13)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,d,ctas", [(8, 2, 128, 0), (8, 2, 64, 5), (64, 2, 128, 3)])
def test_nan_in_places_not_seen(hq, hkv, d, ctas):
    """NaN scale codes past the ends, before the windows, in unused pages, and in the run's own later tokens."""
    c = Case([45, 70, 130], [2, 1, 2], hq=hq, hkv=hkv, d=d, window=20, seed=14)
    used = [set(c.bt[i][c.bt[i] >= 0]) for i in range(3)]
    for s in c.scales:
        for p in range(len(s)):
            if not any(p in u for u in used):
                s[p] = 0x7F
        for i, l in enumerate(c.lens):
            for j in range(len(used[i]) * 16):
                if j >= l or j <= l - c.qlens[i] - 20:
                    s[c.bt[i, j // 16], :, j % 16] = 0xFF
    c.check(*c.run(num_ctas=ctas, min_pages_per_cta=1))
    # the last token of the first and third run: seen by its own row alone
    for i in (0, 2):
        j = c.lens[i] - 1
        for s in c.scales:
            s[c.bt[i, j // 16], 0, j % 16, 1] = 0x7F
    c.check(*c.run(num_ctas=ctas, min_pages_per_cta=1))


def test_nan_seen_is_nan():
    c = Case([300, 40], hq=8, hkv=2, seed=15)
    c.scales[0][c.bt[0, 5], 1, 3, 0] = 0x7F                   # a key of head 1 in the middle
    c.scales[1][c.bt[1, 0], 0, 2, 4] = 0x7F                   # a value group of head 0
    c.check(*c.run())
    c.check(*c.run(num_ctas=9, min_pages_per_cta=1))
    c = Case([3], hq=8, hkv=2, seed=15)
    c.scales[0][c.bt[0, 0]] = 0x7F                            # every key
    c.check(*c.run())


def test_out_of_range_page_is_reported():
    c = Case([40, 40], hq=8, hkv=2, seed=16)
    c.bt[0, 1] = 99
    out, lse = c.run()
    assert binding.paged_attn_device_status() == binding.STATUS_PAGE_RANGE
    c2 = Case([40, 40], hq=8, hkv=2, seed=16)
    wo, wl = c2.run()
    assert torch.equal(out[1], wo[1]) and torch.equal(lse[1], wl[1])


def test_bad_query_ranges_are_reported():
    c = Case([40, 40, 40], [1, 3, 1], hq=8, hkv=2, seed=17)
    c.runs = 2                                                # the second run is longer
    out, lse = c.run()
    assert binding.paged_attn_device_status() == binding.STATUS_QUERY_LEN
    wo, wl = c.want()
    for t in (0, 4):
        assert np.abs(lse[t].cpu().numpy() - wl[t]).max() < 1e-3
    assert (out[1:4] == 7).all() and (lse[1:4] == 7).all()


def test_strided_tensors():
    c = Case([60, 150], [2, 1], hq=8, hkv=2, d=64, seed=18)
    want = c.run()
    dev = c.dev
    nb = dev[1].shape[0]
    kv = torch.zeros(nb, 2, 16, 3, 32, dtype=torch.uint8, device="cuda")
    kv[:, 0, :, :2], kv[:, 1, :, :2] = dev[1], dev[2]
    sc = torch.zeros(nb, 2, 2, 16, 4, dtype=torch.uint8, device="cuda")
    sc[:, 0], sc[:, 1] = dev[3], dev[4]
    q = torch.zeros(3, 8 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    q[:, :512] = dev[0].reshape(3, 512)
    bt = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    bt[:, :dev[5].shape[1]] = dev[5]
    out = torch.full((8, 3, 68), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.full((8, 3), 7.0, device="cuda").t()
    binding.paged_attn_decode_q4(q[:, :512].view(3, 8, 64), kv[:, 0, :, :2], kv[:, 1, :, :2], sc[:, 0], sc[:, 1], bt,
                                 dev[6], dev[7], 2, c.scale, c.k_scale, c.v_scale, out=out[..., :64], lse=lse)
    assert torch.equal(out[..., :64], want[0]) and torch.equal(lse, want[1])
    assert (out[..., 64:] == 7).all()


def test_many_sequences_and_a_long_one():
    r = np.random.default_rng(19)
    c = Case(r.integers(1, 40, 700), hq=4, hkv=1, d=64, seed=19)
    c.check(*c.run())
    c = Case([20000], hq=8, hkv=1, d=64, seed=20)
    c.check(*c.run())
    c = Case(np.ones(8192, dtype=int), hq=1, hkv=1, d=64, seed=21)
    c.check(*c.run())


def test_pages_behind_32_bit_offsets():
    """A page whose bytes lie more than 2^32 from the cache's start."""
    nb = (1 << 32) // (16 * 8 * 64) + 40
    kc = torch.zeros(nb, 16, 8, 64, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(nb, 8, 16, 8, dtype=torch.uint8, device="cuda")
    c = Case([33], hq=8, hkv=8, d=128, seed=22)
    dev = c.on_gpu()
    small = dev[1].shape[0]
    base = nb - small
    kc[base:], ks[base:] = dev[1], dev[3]
    dev[1], dev[3] = kc, ks
    vc = torch.zeros(nb, 16, 8, 64, dtype=torch.uint8, device="cuda")
    vs = torch.zeros(nb, 8, 16, 8, dtype=torch.uint8, device="cuda")
    vc[base:], vs[base:] = dev[2], dev[4]
    dev[2], dev[4], dev[5] = vc, vs, dev[5] + base
    out, lse = binding.paged_attn_decode_q4(*dev, 1, c.scale, c.k_scale, c.v_scale)
    c.check(out, lse)


def test_runs_alike_and_with_its_own_workspace():
    c = Case([500, 3, 260], [2, 1, 3], hq=16, hkv=2, seed=23)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    n = binding.paged_attn_q4_workspace_size(3, 16, 2, 128, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    d = c.run(workspace=ws.data_ptr(), workspace_bytes=n)
    assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])
    with pytest.raises(binding.PagedAttnError) as e:
        c.run(workspace=ws.data_ptr(), workspace_bytes=n - 1)
    assert e.value.status == binding.PA_ERR_WORKSPACE
    binding.paged_attn_q4_reserve(3, 16, 2, 128, 3)


def test_no_lse_and_no_tokens():
    c = Case([50], seed=24)
    want = c.run()
    out, lse = binding.paged_attn_decode_q4(*c.dev, 1, c.scale, c.k_scale, c.v_scale, want_lse=False)
    assert lse is None and torch.equal(out, want[0])
    out, lse = binding.paged_attn_decode_q4(c.dev[0][:0], *c.dev[1:], 1, c.scale, c.k_scale, c.v_scale)
    assert out.shape == (0, 8, 128)


def test_streams_graphs_and_prepared_calls():
    """Two captured graphs replayed at once, and calls on two streams, each with results of their own."""
    cases = [Case([900, 40], hq=8, hkv=2, seed=25), Case([30, 1000], [1, 2], hq=8, hkv=2, seed=26)]
    want = [c.run() for c in cases]
    graphs, outs, streams = [], [], []
    for c in cases:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        call = binding.prepare_decode_q4(*c.dev, c.runs, c.scale, c.k_scale, c.v_scale, options=c.options())
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            direct = binding.paged_attn_decode_q4(*c.dev, c.runs, c.scale, c.k_scale, c.v_scale, options=c.options())
            call()
        graphs.append(g)
        outs.append((direct, (call.out, call.lse), call))
        streams.append(s)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, (a, b, _) in zip(want, outs):
        for got in (a, b):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    got = [[binding.paged_attn_decode_q4(*c.dev, c.runs, c.scale, c.k_scale, c.v_scale, stream=s) for _ in range(5)]
           for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for out, lse in gs:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_write_fork_decode_compact_together():
    """A serving step's calls in a row: rows written, sequences forked, the forks written to and decoded,
    the pool compacted, decoded again."""
    r = np.random.default_rng(27)
    hq, hkv, d, nb = 8, 2, 64, 60
    lens = [37, 64, 5]
    order = r.permutation(nb)
    bt = np.full((6, 8), -1, dtype=np.int32)
    ref = np.zeros(nb, dtype=np.int32)
    at = 0
    for i, l in enumerate(lens):
        k = -(-l // 16)
        bt[i, :k] = order[at:at + k]
        ref[order[at:at + k]] = 1
        at += k
    i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    dbt, dsl, dref = i32(bt), i32(lens + [0, 0, 0]), i32(ref)
    kc, vc = (torch.zeros(nb, 16, hkv, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(nb, hkv, 16, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    caches = [kc, vc, ks, vs]
    g = torch.Generator(device="cuda").manual_seed(27)
    rows = lambda n: torch.randn(n, hkv, d, device="cuda", generator=g).to(torch.bfloat16)
    slot = lambda i, j: int(bt[i, j // 16]) * 16 + j % 16
    slots = [slot(i, j) for i, l in enumerate(lens) for j in range(l)]
    binding.paged_attn_cache_write_q4(rows(len(slots)), rows(len(slots)), i32(slots), *caches, 0.02, 0.02)
    new = order[at:at + 3]
    binding.paged_attn_pages_fork(caches, dbt, dsl, dref, i32([0, 0, 1]), i32([3, 4, 5]), i32(new))
    # the first fork gets a token of its own in its copied page
    bt = dbt.cpu().numpy()
    assert dsl.tolist() == [37, 64, 5, 37, 37, 64]
    own = rows(1)
    binding.paged_attn_cache_write_q4(own, own, i32([int(bt[3, 2]) * 16 + 5]), *caches, 0.02, 0.02)
    dsl[3] += 1
    q = torch.randn(6, hq, d, device="cuda", generator=g).to(torch.bfloat16)
    q[4] = q[0]
    before = binding.paged_attn_decode_q4(q, kc, vc, ks, vs, dbt, dsl, None, 1, None, 0.02, 0.02)
    assert torch.equal(before[0][4], before[0][0])          # an untouched fork answers as its parent
    h = [t.cpu().numpy() for t in (kc, vc, ks, vs)]
    want, wl = cache_q4.decode(q.double().cpu().numpy(), h[:2], h[2:], bt, dsl.cpu().numpy(), None, d ** -0.5, 0.02, 0.02)
    assert np.abs(before[0].double().cpu().numpy() - want).max() < 2e-2
    assert np.abs(before[1].double().cpu().numpy() - wl).max() < 1e-3
    _, num = binding.paged_attn_pages_free(dbt, dsl, dref, i32([1]))
    dsl[1] = 1                                                  # its first page is still its fork's
    page_map, used = binding.paged_attn_pages_compact(caches, dbt, dref)
    assert used.item() + num.item() == nb and int(dbt[5, 0]) == int(page_map[bt[5, 0]])
    dsl[1] = 64                                                 # and so are the others: row 1 reads them still
    after = binding.paged_attn_decode_q4(q, kc, vc, ks, vs, dbt, dsl, None, 1, None, 0.02, 0.02)
    assert torch.equal(after[0], before[0]) and torch.equal(after[1], before[1])
    assert binding.paged_attn_device_status() == 0


def test_give_up_limit_is_not_met():
    c = Case([200, 100], seed=28)
    c.check(*c.run(wait_limit_us=500000))


def test_tensors_off_the_device_are_refused():
    c = Case([20], seed=29)
    dev = c.on_gpu()
    dev[5] = dev[5].cpu()
    with pytest.raises(ValueError):
        binding.paged_attn_decode_q4(*dev, 1, c.scale)


@pytest.mark.parametrize("b,hq,hkv,d,rows,stages", [
    (3000, 8, 8, 64, 1, 8),          # the metadata leaves room for one CTA an SM
    (8192, 1, 1, 64, 32, 8),         # ... for one warp a head
    (8192, 4, 4, 128, 64, 4),        # ... the most shared memory
    (1000, 2, 1, 128, 8, 4), (1000, 2, 2, 64, 20, 8)])
def test_launch_forms(b, hq, hkv, d, rows, stages):
    """Batches whose metadata takes the shared memory of the usual launch (rows: the declared query run)."""
    r = np.random.default_rng(b + rows)
    lens = np.where(r.random(b) < 0.2, r.integers(1, 40, b), 0)
    lens[[7, 500]] = 700, 130
    c = Case(lens, np.ones(b, dtype=np.int64), hq=hq, hkv=hkv, d=d, seed=rows)
    c.runs = rows
    assert binding.paged_attn_q4_plan(b, hq, hkv, d, rows)["num_stages"] == stages
    c.check(*c.run(), status=binding.STATUS_SEQ_LEN)       # sequences of length 0 are reported


@pytest.mark.parametrize("hkv,qlens", [(1, [1, 1, 1]), (1, [2, 2, 1]), (2, [4, 1, 3]), (3, [2, 1, 2]), (4, [4, 4, 4])])
@pytest.mark.parametrize("ctas", [0, 2])
def test_windows_over_shared_heads(hkv, qlens, ctas):
    """Several warps a head, 8 to 32 rows, with pages before, inside and after a window; sinks."""
    c = Case([500, 333, 90], qlens, hq=8 * hkv, hkv=hkv, d=128, window=200, sinks=True, seed=hkv)
    c.check(*c.run(num_ctas=ctas, min_pages_per_cta=1))


@pytest.mark.parametrize("hq,hkv,runs,window", [(32, 8, 5, 0), (32, 8, 8, 40), (64, 8, 8, 0), (16, 4, 16, 0),
                                                (20, 5, 10, 33), (64, 16, 7, 0)])
def test_large_batches_of_many_rows(hq, hkv, runs, window):
    """32 sequences and more with 17 to 64 rows a head of 64 features: the tiles of 32 rows."""
    r = np.random.default_rng(hq + runs)
    lens = r.integers(runs, 300, 37)
    qlens = np.where(r.random(37) < 0.5, runs, r.integers(1, runs, 37))
    c = Case(lens, qlens, hq=hq, hkv=hkv, d=64, window=window, sinks=window > 0, seed=runs)
    c.check(*c.run())


@pytest.mark.parametrize("gain,scale,k_scale", [(2e-38, 1e37, 0.02), (1e-39, 1e37, 0.02), (3e37, 1e-20, 6e-21)])
def test_query_rows_at_the_ends_of_the_range(gain, scale, k_scale):
    """Rows of subnormal elements, and of the largest, with scales that make up for them."""
    c = Case([40, 130], [2, 1], q_gain=gain, scale=scale, k_scale=k_scale, seed=33)
    c.check(*c.run())
