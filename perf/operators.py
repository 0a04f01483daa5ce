"""Cases of the 4-bit KV cache (write and read of rows, decode attention) and of
the cache's page operations (copy, fork and free, compact), for timing.

``run`` computes a case either in its plain form (elementary torch operations)
or, with ``own`` set, with the calls a serving program makes of
``paged_kv_decode_06_gb300.binding``.

The 4-bit cache, per tensor (K or V): codes uint8 [NB, 16, Hkv, D / 2], two
e2m1 codes a byte (the even feature in the low nibble), and group scales uint8
[NB, Hkv, 16, D / 16], one e4m3fn code for 16 consecutive features of a cached
row; a feature's value is e2m1 * e4m3 * (the tensor's one fp32 scale).
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
K_SCALE, V_SCALE = 0.0125, 0.02      # the tensors' fp32 scales (rows of unit variance: group scales near 30 and 20)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest calls: a handful of short sequences, one of a single token; latency is all
        {"name": "decode_short", "op": "decode", "batch": 3, "hq": 8, "hkv": 2, "d": 64, "lo": 1, "hi": 100,
         "runs": 1, "window": 0, "sinks": False, "lens_seed": 1},
        # verification of drafted tokens: ragged runs of 1 to 4, a sliding window with attention sinks
        {"name": "decode_runs", "op": "decode", "batch": 32, "hq": 64, "hkv": 8, "d": 128, "lo": 1024, "hi": 16384,
         "runs": 4, "window": 4096, "sinks": True, "lens_seed": 2},
        # one user with a long context: the walk of one sequence split over the whole device
        {"name": "decode_long", "op": "decode", "batch": 1, "hq": 64, "hkv": 8, "d": 64, "lo": 32768, "hi": 32768,
         "runs": 1, "window": 0, "sinks": False, "lens_seed": 3},
        # a full serving batch with log-uniform lengths, single tokens
        {"name": "decode_batch", "op": "decode", "batch": 256, "hq": 32, "hkv": 8, "d": 128, "lo": 128, "hi": 8192,
         "runs": 1, "window": 0, "sinks": False, "lens_seed": 4},
        # the rows of one decode step (a token a sequence) written, then read back
        {"name": "rows_step", "op": "rows", "tokens": 64, "hkv": 8, "d": 128, "pool": 4096},
        # a prefill chunk
        {"name": "rows_chunk", "op": "rows", "tokens": 16384, "hkv": 8, "d": 128, "pool": 1200},
        # a few pages of one bf16 layer: a prefix made private
        {"name": "copy_few", "op": "copy", "pages": 5, "pool": 256, "layers": 1, "kind": "bf16", "hkv": 8, "d": 128},
        # many pages of several 4-bit layers: a batch of prompts duplicated
        {"name": "copy_many", "op": "copy", "pages": 2048, "pool": 6000, "layers": 8, "kind": "q4", "hkv": 8,
         "d": 128},
        # a few short sequences branched, then the branches dropped
        {"name": "branch_few", "op": "branch", "rows": 16, "forks": 4, "lo": 1, "hi": 300, "layers": 1, "kind": "q4",
         "hkv": 2, "d": 64, "lens_seed": 5},
        # a batch branched (two candidates a sequence), then the branches dropped
        {"name": "branch_many", "op": "branch", "rows": 512, "forks": 256, "lo": 512, "hi": 4096, "layers": 2,
         "kind": "q4", "hkv": 8, "d": 128, "lens_seed": 6},
        # a small pool compacted
        {"name": "compact_few", "op": "compact", "pool": 100, "used": 0.5, "batch": 6, "layers": 1, "kind": "bf16",
         "hkv": 2, "d": 64},
        # a large fragmented pool compacted before part of it is given back
        {"name": "compact_many", "op": "compact", "pool": 32768, "used": 0.6, "batch": 128, "layers": 2, "kind": "q4",
         "hkv": 8, "d": 128},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "rows", "copy", "branch", "compact"])
    if op == "decode":
        hkv = rng.choice([1, 2, 3, 4, 5, 8, 10])
        runs = rng.choice([1, 1, 1, 2, 3, 4, 7])
        g = rng.choice([x for x in (1, 2, 3, 4, 5, 7, 8, 16, 32, 64) if x * runs <= 64])
        d = rng.choice([64, 128])
        batch = _logint(rng, 1, 256)
        # 6e8 cached values a tensor at most
        hi = _logint(rng, 1, max(1, min(100000, int(6e8 / (batch * hkv * d)))))
        lo = rng.randint(1, hi)
        return {"op": op, "batch": batch, "hq": g * hkv, "hkv": hkv, "d": d, "lo": lo, "hi": hi, "runs": runs,
                "window": rng.choice([0, 0, 0, _logint(rng, 1, 8192)]), "sinks": rng.random() < 0.3,
                "lens_seed": rng.randrange(1 << 30)}
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rows":
        tokens = _logint(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "hkv": hkv, "d": 16 * rng.choice([1, 2, 3, 4, 5, 6, 8]),
                "pool": tokens // PAGE + _logint(rng, 1, 1000)}
    layers, kind, d = rng.randint(1, 8), rng.choice(["bf16", "q4"]), rng.choice([64, 128])
    per_page = _page_bytes({"layers": layers, "kind": kind, "hkv": hkv, "d": d})
    if op == "copy":
        pages = _logint(rng, 1, max(1, min(4096, int(2.5e8 / per_page))))
        return {"op": op, "pages": pages, "pool": 2 * pages + rng.randint(0, 500), "layers": layers, "kind": kind,
                "hkv": hkv, "d": d}
    if op == "branch":
        rows = 2 * _logint(rng, 1, 256)
        hi = _logint(rng, 1, max(1, min(8192, int(16 * 1.0e9 / (per_page * rows)))))
        return {"op": op, "rows": rows, "forks": rng.randint(1, rows // 2), "lo": rng.randint(1, hi), "hi": hi,
                "layers": layers, "kind": kind, "hkv": hkv, "d": d, "lens_seed": rng.randrange(1 << 30)}
    return {"op": op, "pool": _logint(rng, 1, max(1, min(65536, int(1.1e9 / per_page)))),
            "used": rng.uniform(0.05, 0.95), "batch": _logint(rng, 1, 256), "layers": layers, "kind": kind,
            "hkv": hkv, "d": d}


# ----------------------------------------------------------- sizes of a case

def _lens(case):
    """(cached tokens, query tokens) of each sequence; the cached tokens include the run."""
    r = np.random.default_rng(case["lens_seed"])
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    ln = np.floor(np.exp(r.uniform(math.log(lo), math.log(hi + 1), b))).astype(np.int64).clip(lo, hi)
    qn = r.integers(1, case["runs"] + 1, b)
    if case["runs"] > 1:
        qn[0] = case["runs"]
    return np.maximum(ln, qn), qn


def _branch_lens(case):
    r = np.random.default_rng(case["lens_seed"])
    return r.integers(case["lo"], case["hi"] + 1, case["rows"] // 2)


def _branch_parents(case):
    r = np.random.default_rng(case["lens_seed"] + 1)
    return r.integers(0, case["rows"] // 2, case["forks"])


def _compact_used(case):
    """Pages in use of a fragmented pool, and how many each table row holds (by the case's sizes alone)."""
    n = max(1, int(round(case["used"] * case["pool"])))
    r = np.random.default_rng(case["pool"] * 1000 + n)
    used = np.zeros(case["pool"], dtype=bool)
    used[r.permutation(case["pool"])[:n]] = True
    cut = np.sort(r.integers(0, n + 1, case["batch"] - 1))
    return used, np.diff(np.concatenate([[0], cut, [n]]))


def _page_bytes(case):
    per = case["hkv"] * PAGE * case["d"]
    return case["layers"] * 2 * (2 * per if case["kind"] == "bf16" else per // 2 + per // 16)


def work(case):
    op = case["op"]
    if op == "decode":
        ln, qn = _lens(case)
        w = case["window"]
        seen = rows = 0        # cached tokens some query row sees; (row, key) pairs
        for l, q in zip(ln.tolist(), qn.tolist()):
            seen += min(l, w + q - 1) if w else l
            rows += sum(min(l - q + r + 1, w) if w else l - q + r + 1 for r in range(q))
        t, hq, hkv, d = int(qn.sum()), case["hq"], case["hkv"], case["d"]
        kv = seen * hkv * 2 * (d // 2 + d // 16)
        return {"bytes": kv + t * hq * (4 * d + 4) + 4 * (seen // PAGE + 2 * len(ln)), "flops": 4 * d * hq * rows}
    if op == "rows":
        n = case["tokens"] * case["hkv"] * case["d"] * 2
        # written: bf16 rows read, codes and scales written; read: the reverse
        return {"bytes": 2 * (2 * n + n // 2 + n // 16) + 8 * case["tokens"], "flops": 4 * n}
    if op == "copy":
        return {"bytes": case["pages"] * (2 * _page_bytes(case) + 8), "flops": 0}
    if op == "branch":
        ln = _branch_lens(case)[_branch_parents(case)]
        part = int((ln % PAGE != 0).sum())
        pages = int((-(-ln // PAGE)).sum())
        pool = _branch_pool(case)
        # fork: table rows read and written, counts updated, one page a ragged fork copied;
        # free: rows read, counts updated, the pool's counts read and its free list written
        return {"bytes": part * 2 * _page_bytes(case) + 4 * (7 * pages + 2 * pool), "flops": 0}
    used, _ = _compact_used(case)
    moved = int(used[int(used.sum()):].sum())
    return {"bytes": moved * 2 * _page_bytes(case) + 4 * (3 * case["pool"] + 4 * int(used.sum())), "flops": 0}


def _branch_pool(case):
    pages = int((-(-_branch_lens(case) // PAGE)).sum())
    return pages + case["forks"] + 7


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ieee(x, divisor):
    """x / divisor with a device tensor as divisor: the IEEE fp32 quotient."""
    return x / torch.full((), divisor, dtype=torch.float32, device=x.device)


def _quantise(x, tensor_scale):
    """Rows x (float32 [..., D]) -> (packed codes [..., D / 2], scale codes [..., D / 16])."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    six = float(np.float32(6.0) * np.float32(tensor_scale))
    s8 = _ieee(g.abs().amax(-1), six).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s8.float() * torch.full((), tensor_scale, dtype=torch.float32, device=x.device)).unsqueeze(-1)
    y = torch.where(d > 0, g / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(g))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * ((g < 0) & (d > 0))
    code = code.to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _fill(nb, hkv, d, tensor_scale, gen):
    """One tensor of a 4-bit cache holding rows of unit variance."""
    codes = torch.empty(nb, PAGE, hkv, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(nb, hkv, PAGE, d // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (PAGE * hkv * d))
    for a in range(0, nb, step):
        n = min(nb, a + step) - a
        c, s = _quantise(torch.randn(n, PAGE, hkv, d, generator=gen, device="cuda"), tensor_scale)
        codes[a:a + n] = c
        scales[a:a + n] = s.permute(0, 2, 1, 3)
    return codes, scales


def _layers(case, nb, gen):
    """The page tensors of some layers: K and V, and for 4-bit caches their group scales."""
    hkv, d, out = case["hkv"], case["d"], []
    for _ in range(case["layers"]):
        if case["kind"] == "bf16":
            out += [torch.randn(nb, PAGE, hkv, d, generator=gen, device="cuda", dtype=torch.bfloat16)
                    for _ in range(2)]
        else:
            for _ in range(2):
                out.append(torch.randint(0, 256, (nb, PAGE, hkv, d // 2), generator=gen, device="cuda",
                                         dtype=torch.uint8))
                out.append(torch.randint(0, 127, (nb, hkv, PAGE, d // 16), generator=gen, device="cuda",
                                         dtype=torch.uint8))
    return out


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _tables(pages, width, order):
    """Block-table rows holding consecutive runs of `order`, -1 past a row's end."""
    bt = np.full((len(pages), width), -1, dtype=np.int64)
    at = 0
    for i, n in enumerate(pages):
        bt[i, :n] = order[at:at + n]
        at += n
    return bt


def prepare(case, seed):
    op, gen, r = case["op"], _gen(seed), np.random.default_rng(seed)
    st = {"op": op, "case": case}
    if op == "decode":
        ln, qn = _lens(case)
        pages = -(-ln // PAGE)
        nb = int(math.ceil(1.1 * pages.sum()))
        st["k"], st["ks"] = _fill(nb, case["hkv"], case["d"], K_SCALE, gen)
        st["v"], st["vs"] = _fill(nb, case["hkv"], case["d"], V_SCALE, gen)
        st["bt"] = _i32(_tables(pages, int(pages.max()), r.permutation(nb)))
        st["lens"], st["qlens"] = ln.tolist(), qn.tolist()      # the scheduler's host copies
        st["sl"] = _i32(ln)
        st["qsl"] = _i32(np.concatenate([[0], np.cumsum(qn)])) if case["runs"] > 1 else None
        t = int(qn.sum())
        st["q"] = torch.randn(t, case["hq"], case["d"], generator=gen, device="cuda").to(torch.bfloat16)
        st["sinks"] = torch.randn(case["hq"], generator=gen, device="cuda") if case["sinks"] else None
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(t, case["hq"], device="cuda")
        if own:
            from paged_kv_decode_06_gb300 import binding
            opts = None
            if case["window"] or st["sinks"] is not None:
                opts = binding.make_options(sliding_window=case["window"], sinks=st["sinks"])
            st["call"] = binding.prepare_decode_q4(
                st["q"], st["k"], st["v"], st["ks"], st["vs"], st["bt"], st["sl"], st["qsl"], case["runs"],
                case["d"] ** -0.5, K_SCALE, V_SCALE, out=st["out"], lse=st["lse"], options=opts)
    elif op == "rows":
        t, hkv, d, nb = case["tokens"], case["hkv"], case["d"], case["pool"]
        for name in ("key", "value"):
            # rows of different size, as tokens have
            x = torch.randn(t, hkv, d, generator=gen, device="cuda")
            st[name] = (x * torch.exp(0.5 * torch.randn(t, hkv, 1, generator=gen, device="cuda"))).to(torch.bfloat16)
            st[name + "_out"] = torch.zeros_like(st[name])
        slots = r.permutation(nb * PAGE)[:t]
        slots[r.random(t) < 0.02] = -1                          # padding tokens
        st["slots"] = _i32(slots)
        st["k"], st["ks"] = _fill(nb, hkv, d, K_SCALE, gen)
        st["v"], st["vs"] = _fill(nb, hkv, d, V_SCALE, gen)
    elif op == "copy":
        nb, n = case["pool"], case["pages"]
        perm = r.permutation(nb)
        st["caches"] = _layers(case, nb, gen)
        st["dst"] = _i32(perm[:n])
        st["src"] = _i32(perm[n + r.integers(0, nb - n, n)])    # a page may be copied to several
    elif op == "branch":
        ln = _branch_lens(case)
        pages, half = -(-ln // PAGE), case["rows"] // 2
        nb = _branch_pool(case)
        order = r.permutation(nb)
        bt = np.full((case["rows"], int(pages.max())), -1, dtype=np.int64)
        place = r.permutation(case["rows"])                     # rows of the table: parents, then free ones
        bt[place[:half]] = _tables(pages, int(pages.max()), order)
        ref = np.zeros(nb, dtype=np.int64)
        ref[order[:pages.sum()]] = 1
        lens = np.zeros(case["rows"], dtype=np.int64)
        lens[place[:half]] = ln
        st["caches"] = _layers(case, nb, gen)
        st["bt"], st["sl"], st["ref"] = _i32(bt), _i32(lens), _i32(ref)
        st["parents"] = _i32(place[_branch_parents(case)])
        st["children"] = _i32(place[half:half + case["forks"]])
        st["new"] = _i32(order[pages.sum():pages.sum() + case["forks"]])
        st["free"] = torch.empty(nb, dtype=torch.int32, device="cuda")
        st["nfree"] = torch.empty(1, dtype=torch.int32, device="cuda")
    else:
        nb = case["pool"]
        used, pages = _compact_used(case)
        ids = r.permutation(np.flatnonzero(used))
        bt = _tables(pages, max(1, int(pages.max())), ids)
        ref = np.zeros(nb, dtype=np.int64)
        ref[ids] = r.integers(1, 4, len(ids))                   # some pages have holders outside the tables
        st["caches"] = _layers(case, nb, gen)
        # the scheduler's tables of this step, and the buffers they are compacted in
        st["bt0"], st["ref0"] = _i32(bt), _i32(ref)
        st["bt"], st["ref"] = torch.empty_like(st["bt0"]), torch.empty_like(st["ref0"])
        st["map"] = torch.empty(nb, dtype=torch.int32, device="cuda")
        st["nused"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

_LUT = {}


def _pairs(device):
    """float32 [256, 2]: the two e2m1 values of a code byte."""
    if device not in _LUT:
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=device)
        b = torch.arange(256, device=device)
        _LUT[device] = torch.stack([v[b & 15], v[b >> 4]], -1)
    return _LUT[device]


def _values(codes, scales, tensor_scale):
    """Codes [..., D / 2] and scale codes [..., D / 16] -> float32 [..., D]."""
    x = _pairs(codes.device)[codes.to(torch.int32)].flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2) * tensor_scale


def _plain_decode(st):
    c = st["case"]
    hq, hkv, d, w = c["hq"], c["hkv"], c["d"], c["window"]
    g, t0 = hq // hkv, 0
    out, lse = torch.empty_like(st["q"]), torch.empty_like(st["lse"])
    for i, (l, qn) in enumerate(zip(st["lens"], st["qlens"])):
        pages = st["bt"][i, :-(-l // PAGE)].long()
        k = _values(st["k"][pages], st["ks"][pages].transpose(1, 2), K_SCALE).reshape(-1, hkv, d)[:l]
        v = _values(st["v"][pages], st["vs"][pages].transpose(1, 2), V_SCALE).reshape(-1, hkv, d)[:l]
        q = st["q"][t0:t0 + qn].float().reshape(qn, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, qn * g, d)
        s = torch.matmul(q, k.permute(1, 2, 0)) * d ** -0.5
        pos = torch.arange(l - qn, l, device=s.device).repeat_interleave(g).unsqueeze(1)
        j = torch.arange(l, device=s.device).unsqueeze(0)
        hide = (j > pos) | (j <= pos - w) if w else j > pos
        s = s.masked_fill(hide, -math.inf)
        m = s.amax(-1, keepdim=True)
        if st["sinks"] is not None:
            sink = st["sinks"].reshape(hkv, 1, g).expand(hkv, qn, g).reshape(hkv, qn * g, 1)
            m = torch.maximum(m, sink)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        if st["sinks"] is not None:
            z = z + torch.exp(sink - m)
        o = torch.matmul(e, v.transpose(0, 1)) / z
        out[t0:t0 + qn] = o.reshape(hkv, qn, g, d).permute(1, 0, 2, 3).reshape(qn, hq, d).to(torch.bfloat16)
        lse[t0:t0 + qn] = (m + torch.log(z)).reshape(hkv, qn, g).permute(1, 0, 2).reshape(qn, hq)
        t0 += qn
    return out, lse


def _plain_rows(st):
    slots = st["slots"].long()
    live = (slots >= 0).nonzero().squeeze(1)
    page, off = slots[live] // PAGE, slots[live] % PAGE
    for x, codes, scales, ts in ((st["key"], st["k"], st["ks"], K_SCALE), (st["value"], st["v"], st["vs"], V_SCALE)):
        c, s = _quantise(x[live].float(), ts)
        codes[page, off] = c
        scales[page, :, off] = s
    st["key_out"][live] = _values(st["k"][page, off], st["ks"][page, :, off], K_SCALE).to(torch.bfloat16)
    st["value_out"][live] = _values(st["v"][page, off], st["vs"][page, :, off], V_SCALE).to(torch.bfloat16)


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for c in st["caches"]:
        c[dst] = c[src]


def _plain_branch(st):
    bt, sl, ref = st["bt"], st["sl"], st["ref"]
    par, chi, new = st["parents"].long(), st["children"].long(), st["new"].long()
    col = torch.arange(bt.shape[1], device=bt.device).unsqueeze(0)
    # fork: full pages shared, the partial last page copied to the child's own
    ln = sl[par].long()
    full, part = (ln // PAGE).unsqueeze(1), (ln % PAGE > 0).unsqueeze(1)
    rows = bt[par].long()
    last = torch.gather(rows, 1, full.clamp(max=bt.shape[1] - 1)).squeeze(1)
    mine = torch.where(col < full, rows, torch.where((col == full) & part, new.unsqueeze(1), bt[chi].long()))
    take = part.squeeze(1).nonzero().squeeze(1)
    for c in st["caches"]:
        c[new[take]] = c[last[take]]
    ref.index_add_(0, new[take], torch.ones_like(new[take], dtype=torch.int32))
    shared = rows[(col < full).expand_as(rows)]
    ref.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    bt[chi] = mine.int()
    sl[chi] = ln.int()
    # free the same rows, then list the free pages in ascending order
    held = (sl[chi].long() + PAGE - 1) // PAGE
    gone = bt[chi].long()[(col < held.unsqueeze(1)).expand(len(chi), -1)]
    ref.index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    sl[chi] = 0
    free = (ref == 0).nonzero().squeeze(1)
    st["free"].fill_(-1)
    st["free"][:len(free)] = free.int()
    st["nfree"].fill_(len(free))


def _plain_compact(st):
    ref, bt, nb = st["ref"], st["bt"], st["ref"].numel()
    ids = torch.arange(nb, device=ref.device)
    used = ref > 0
    n = used.sum()
    src = (used & (ids >= n)).nonzero().squeeze(1)
    dst = (~used & (ids < n)).nonzero().squeeze(1)
    for c in st["caches"]:
        c[dst] = c[src]
    st["map"].copy_(torch.where(used, ids, -1))
    st["map"][src] = dst.int()
    ref[dst] = ref[src]
    ref[src] = 0
    there = st["map"][bt.long().clamp(0, nb - 1)]
    bt.copy_(torch.where((bt >= 0) & (bt < nb) & (there >= 0), there, bt))
    st["nused"].copy_(n.reshape(1))


# ------------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        from paged_kv_decode_06_gb300 import binding as b
    if op == "decode":
        return st["call"]() if own else _plain_decode(st)
    if op == "rows":
        if own:
            b.paged_attn_cache_write_q4(st["key"], st["value"], st["slots"], st["k"], st["v"], st["ks"], st["vs"],
                                        K_SCALE, V_SCALE)
            b.paged_attn_cache_read_q4(st["slots"], st["k"], st["v"], st["ks"], st["vs"], st["key_out"],
                                       st["value_out"], K_SCALE, V_SCALE)
        else:
            _plain_rows(st)
        return st["key_out"], st["value_out"]
    if op == "copy":
        if own:
            b.paged_attn_pages_copy(st["caches"], st["src"], st["dst"])
        else:
            _plain_copy(st)
        return _words(st["caches"])
    if op == "branch":
        if own:
            b.paged_attn_pages_fork(st["caches"], st["bt"], st["sl"], st["ref"], st["parents"], st["children"],
                                    st["new"])
            b.paged_attn_pages_free(st["bt"], st["sl"], st["ref"], st["children"], st["free"], st["nfree"])
        else:
            _plain_branch(st)
        return [st["bt"], st["sl"], st["ref"], st["free"], st["nfree"]] + _words(st["caches"])
    st["bt"].copy_(st["bt0"])
    st["ref"].copy_(st["ref0"])
    if own:
        b.paged_attn_pages_compact(st["caches"], st["bt"], st["ref"], st["map"], st["nused"])
    else:
        _plain_compact(st)
    return [st["bt"], st["ref"], st["map"], st["nused"]] + _words(st["caches"])


def _words(caches):
    """Page contents as they are moved: opaque 32-bit words."""
    return [c.view(torch.int32) for c in caches]


# -------------------------------------------------- the definitions in 64 bits

def _e4m3_value(code):
    """Values of e4m3fn codes from the format's definition: bias 7, subnormals at 2^-9."""
    code = code.long()
    e, m = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e == 0, m / 512.0, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    return torch.where(code >= 128, -mag, mag)


def _e2m1_value(code):
    """Values of e2m1 codes: sign, two exponent bits (bias 1), one mantissa bit."""
    code = code.long()
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2.0, (1.0 + m / 2.0) * torch.exp2((e - 1).double()))
    return torch.where(code >= 8, -mag, mag)


def _stored(codes, scales, tensor_scale):
    x = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    x[..., 0::2] = _e2m1_value(codes & 15)
    x[..., 1::2] = _e2m1_value(codes >> 4)
    return x * _e4m3_value(scales).repeat_interleave(16, -1) * float(np.float32(tensor_scale))


def _exact_decode(case, st):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for i, (l, qn) in enumerate(zip(st["lens"], st["qlens"])):
        slots = torch.arange(l, device="cuda")
        page, off = st["bt"][i].long()[slots // PAGE], slots % PAGE
        k = _stored(st["k"][page, off], st["ks"][page, :, off], K_SCALE)
        v = _stored(st["v"][page, off], st["vs"][page, :, off], V_SCALE)
        for r in range(qn):
            last = l - qn + r
            first = max(0, last - case["window"] + 1) if case["window"] else 0
            q = st["q"][t].double().reshape(hkv, g, d)
            s = torch.einsum("hgd,jhd->hgj", q, k[first:last + 1]) / math.sqrt(d)
            if st["sinks"] is not None:
                s = torch.cat([s, st["sinks"].double().reshape(hkv, g, 1)], -1)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z.unsqueeze(-1))[..., :last + 1 - first]
            out[t] = torch.einsum("hgj,jhd->hgd", p, v[first:last + 1]).reshape(hq, d)
            lse[t] = z.reshape(hq)
            t += 1
    return out, lse


def _nearest(x, grid):
    """Nearest entry of an ascending grid (ties to the even index), its last entry beyond it."""
    hi = torch.searchsorted(grid, x).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - grid[lo], grid[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), grid[lo], grid[hi])


def _exact_rows(x, slots, tensor_scale):
    """Write and read of rows: group scale e4m3(amax / (6 s)), code e2m1(x / (scale s)), value
    code * scale * s; the two quotients and the products 6 s and scale s are fp32 by definition."""
    n = x.shape[-1] // 16
    g = x.double().reshape(*x.shape[:-1], n, 16)
    ts = np.float32(tensor_scale)
    e4 = _e4m3_value(torch.arange(127, device=x.device))
    e2 = _e2m1_value(torch.arange(8, device=x.device))
    amax = g.abs().amax(-1)
    scale = _nearest((amax / float(np.float32(6) * ts)).float().double(), e4)
    step = (scale * float(ts)).float().double().unsqueeze(-1)
    quot = (g.abs() / step).float().double()
    code = torch.where(step > 0, _nearest(torch.nan_to_num(quot, posinf=1e30), e2), torch.zeros_like(g))
    val = torch.sign(g) * code * scale.unsqueeze(-1) * float(ts)
    return torch.where((slots >= 0).reshape(-1, 1, 1), val.reshape(x.shape), torch.zeros_like(x, dtype=torch.float64))


def _exact_branch(case, st):
    """Fork and free leave the tables, lengths and counts as they were but for the children's rows."""
    bt, sl, ref = st["bt"].cpu().numpy().copy(), st["sl"].cpu().numpy(), st["ref"].cpu().numpy()
    for p, c, n in zip(st["parents"].tolist(), st["children"].tolist(), st["new"].tolist()):
        full, rest = divmod(int(sl[p]), PAGE)
        bt[c, :full] = bt[p, :full]
        if rest:
            bt[c, full] = n
    free = [p for p in range(len(ref)) if ref[p] == 0]
    return [bt, sl, ref, np.array(free + [-1] * (len(ref) - len(free))), np.array([len(free)])]


def _exact_compact(case, st):
    bt, ref = st["bt0"].cpu().numpy(), st["ref0"].cpu().numpy()
    n = sum(1 for x in ref if x > 0)
    holes = [p for p in range(n) if ref[p] <= 0]
    new, refs = np.full(len(ref), -1), np.zeros(len(ref), dtype=np.int64)
    for p in range(len(ref)):
        if ref[p] > 0:
            new[p] = p if p < n else holes.pop(0)
            refs[new[p]] = ref[p]
    there = np.where(bt >= 0, new[np.maximum(bt, 0)], -1)
    return [np.where(there >= 0, there, bt), refs, new, np.array([n])]


def exact(case, seed):
    op, st = case["op"], prepare(case, seed)
    if op == "decode":
        return _exact_decode(case, st)
    if op == "rows":
        return (_exact_rows(st["key"], st["slots"], K_SCALE), _exact_rows(st["value"], st["slots"], V_SCALE))
    if op == "copy":
        at = torch.arange(case["pool"], device="cuda")          # where each page's contents come from
        at[st["dst"].long()] = st["src"].long()
        return [w[at] for w in _words(st["caches"])]
    ints = _exact_branch(case, st) if op == "branch" else _exact_compact(case, st)
    return [torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda() for x in ints] + \
        [None] * len(st["caches"])
