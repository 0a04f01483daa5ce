"""Cases of a decode step's rotary positions with the cache write, of decode
attention over a sliding window with first tokens that stay visible, and of
decode attention for a batch that shares prefixes, for timing.

``run`` computes a case either in its plain form (elementary torch operations)
or, with ``own`` set, with the calls a serving program makes of
``paged_kv_decode_06_gb300.binding``.

rope    query and key rows rotated by the angles of their tokens' positions
        (one to three axes: time, height, width), the query written out, key and
        value rows written to their slots of the paged caches (bf16, or e4m3fn
        codes of x / scale).
window  a query at position p sees the keys j <= p with j > p - window or
        j < first.
shared  the sequences of a group hold the same pages for their first tokens;
        those are attended once for all of the group's queries.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
K_SCALE, V_SCALE = 0.05, 0.04       # fp8 caches: a value is code * scale
THETA = 10000.0


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: a token a sequence, three axes in blocks, a bf16 cache; latency is all
        {"name": "rope_step", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 3,
         "order": "blocks", "pairs": "halves", "kv": "bf16", "pool": 1100},
        # a ragged chunk of text: one axis, neighbouring features paired, part of the head rotated
        {"name": "rope_ragged", "op": "rope", "tokens": 777, "hq": 10, "hkv": 5, "d": 96, "rot": 48, "axes": 1,
         "order": "blocks", "pairs": "neighbours", "kv": "bf16", "pool": 300},
        # a prefill chunk of images and text: three axes in turn, an fp8 cache
        {"name": "rope_chunk", "op": "rope", "tokens": 16384, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 3,
         "order": "turns", "pairs": "halves", "kv": "fp8", "pool": 1200},
        # a few short sequences, some shorter than the window
        {"name": "window_short", "op": "window", "batch": 5, "hq": 8, "hkv": 2, "d": 64, "lo": 1, "hi": 300, "runs": 1,
         "window": 64, "first": 4, "kv": "bf16", "lens_seed": 1},
        # one user with a very long dialogue
        {"name": "window_long", "op": "window", "batch": 1, "hq": 64, "hkv": 8, "d": 64, "lo": 131072, "hi": 131072,
         "runs": 1, "window": 32768, "first": 16, "kv": "bf16", "lens_seed": 2},
        # verification of drafted tokens over an fp8 cache
        {"name": "window_runs", "op": "window", "batch": 32, "hq": 64, "hkv": 8, "d": 128, "lo": 1024, "hi": 16384,
         "runs": 4, "window": 1000, "first": 70, "kv": "fp8", "lens_seed": 3},
        # a serving batch of ragged dialogues
        {"name": "window_batch", "op": "window", "batch": 96, "hq": 32, "hkv": 8, "d": 128, "lo": 1024, "hi": 16384,
         "runs": 1, "window": 4096, "first": 4, "kv": "bf16", "lens_seed": 4},
        # a few sequences with a short instruction in common
        {"name": "shared_short", "op": "shared", "groups": 1, "batch": 4, "hq": 8, "hkv": 2, "d": 64, "plo": 100,
         "phi": 100, "lo": 1, "hi": 40, "runs": 1, "kv": "bf16", "lens_seed": 5},
        # several candidate answers about one long document
        {"name": "shared_document", "op": "shared", "groups": 1, "batch": 8, "hq": 64, "hkv": 8, "d": 64,
         "plo": 65536, "phi": 65536, "lo": 1, "hi": 500, "runs": 1, "kv": "bf16", "lens_seed": 6},
        # a serving batch behind one instruction text
        {"name": "shared_batch", "op": "shared", "groups": 1, "batch": 64, "hq": 32, "hkv": 8, "d": 128, "plo": 8192,
         "phi": 8192, "lo": 16, "hi": 512, "runs": 1, "kv": "bf16", "lens_seed": 7},
        # several instruction texts, drafted tokens, an fp8 cache
        {"name": "shared_groups", "op": "shared", "groups": 5, "batch": 96, "hq": 64, "hkv": 8, "d": 128, "plo": 512,
         "phi": 16384, "lo": 4, "hi": 700, "runs": 3, "kv": "fp8", "lens_seed": 8},
        # the full batch behind one long text
        {"name": "shared_large", "op": "shared", "groups": 1, "batch": 256, "hq": 64, "hkv": 8, "d": 128,
         "plo": 32768, "phi": 32768, "lo": 16, "hi": 1024, "runs": 1, "kv": "bf16", "lens_seed": 9},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "window", "shared", "shared"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 10])
    if op == "rope":
        d = 16 * rng.choice([2, 3, 4, 5, 6, 8, 10, 12, 16])
        rot = rng.choice([d, d, d // 2, d // 4])
        g = rng.choice([1, 2, 3, 4, 7, 8])
        tokens = _logint(rng, 1, max(1, min(16384, int(8e7 / ((g + 2) * hkv * d)))))
        axes = rng.choice([1, 2, 3])
        return {"op": op, "tokens": tokens, "hq": g * hkv, "hkv": hkv, "d": d, "rot": max(4 * axes, rot - rot % 4),
                "axes": axes, "order": rng.choice(["blocks", "turns"]), "pairs": rng.choice(["halves", "neighbours"]),
                "kv": rng.choice(["bf16", "fp8"]), "pool": tokens // PAGE + _logint(rng, 1, 1000)}
    runs = rng.choice([1, 1, 1, 2, 3, 4, 7])
    g = rng.choice([x for x in (1, 2, 3, 4, 5, 7, 8, 16, 32, 64) if x * runs <= 64])
    d, kv = rng.choice([64, 128]), rng.choice(["bf16", "fp8"])
    case = {"op": op, "hq": g * hkv, "hkv": hkv, "d": d, "runs": runs, "kv": kv, "lens_seed": rng.randrange(1 << 30)}
    if op == "window":
        batch = _logint(rng, 1, 256)
        hi = _logint(rng, 1, max(1, min(131072, int(1e9 / (batch * hkv * d)))))      # 1e9 cached values a tensor at most
        lo = rng.randint(1, hi)
        most = int(min(2.5e8 / (batch * hkv * d), 2.5e11 / (4 * batch * case["hq"] * d * runs)))
        return {**case, "batch": batch, "lo": lo, "hi": hi, "window": _logint(rng, 1, max(1, min(32768, most))),
                "first": rng.choice([0, 1, 4, 16, _logint(rng, 1, 300)])}
    batch = _logint(rng, 1, 256)
    groups = rng.randint(1, min(8, batch))
    phi = _logint(rng, 16, max(16, min(65536, int(3e11 / (4 * d * case["hq"] * runs * batch)))))
    hi = _logint(rng, 1, max(1, min(1024, int(4e8 / (batch * hkv * d)))))
    return {**case, "groups": groups, "batch": batch, "plo": rng.randint(1, phi), "phi": phi, "lo": rng.randint(1, hi),
            "hi": hi}


# ----------------------------------------------------------- sizes of a case

def _lens(case):
    """(tokens of its own, query tokens) of each sequence; the first include the run."""
    r = np.random.default_rng(case["lens_seed"])
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    ln = np.floor(np.exp(r.uniform(math.log(lo), math.log(hi + 1), b))).astype(np.int64).clip(lo, hi)
    qn = r.integers(1, case["runs"] + 1, b)
    if case["runs"] > 1:
        qn[0] = case["runs"]
    return np.maximum(ln, qn), qn


def _groups(case):
    """(first sequence of each group and the end, tokens that each group's sequences have in common)."""
    r = np.random.default_rng(case["lens_seed"] + 1)
    n = case["groups"]
    cut = np.sort(r.permutation(np.arange(1, case["batch"]))[:n - 1]) if n > 1 else np.zeros(0, dtype=np.int64)
    lens = np.floor(np.exp(r.uniform(math.log(case["plo"]), math.log(case["phi"] + 1), n))).astype(np.int64)
    return np.concatenate([[0], cut, [case["batch"]]]), lens.clip(case["plo"], case["phi"])


def _pair_axis(case):
    """The axis of each rotated pair of features: blocks of pairs an axis, or the axes in turn."""
    n, a = case["rot"] // 2, case["axes"]
    if case["order"] == "turns":
        return [i % a for i in range(n)]
    return [min(i * a // n, a - 1) for i in range(n)]


def work(case):
    hq, hkv, d, es = case["hq"], case["hkv"], case["d"], 2 if case["kv"] == "bf16" else 1
    if case["op"] == "rope":
        t = case["tokens"]
        # query read and written, key and value read, cache rows written, one angle row a token and axis
        return {"bytes": t * d * (4 * hq + hkv * (4 + 2 * es)) + t * 4 * (case["axes"] + 1 + case["rot"]),
                "flops": 3 * t * case["rot"] * (hq + hkv)}
    ln, qn = _lens(case)
    io = int(qn.sum()) * hq * (4 * d + 4)
    if case["op"] == "window":
        w, f = case["window"], case["first"]
        seen = rows = 0                                   # keys that some row sees; (row, key) pairs
        for l, q in zip(ln.tolist(), qn.tolist()):
            seen += min(l, f + w + q - 1)
            rows += sum(min(l - q + r + 1, w + min(f, max(0, l - q + r + 1 - w))) for r in range(q))
        return {"bytes": seen * hkv * 2 * d * es + io + 4 * (seen // PAGE + 2 * len(ln)), "flops": 4 * d * hq * rows}
    at, pre = _groups(case)
    rows = 0
    for g in range(case["groups"]):
        for i in range(at[g], at[g + 1]):
            rows += int(qn[i]) * int(pre[g] + ln[i] - qn[i]) + int(qn[i]) * (int(qn[i]) + 1) // 2
    seen = int(pre.sum() + ln.sum())
    return {"bytes": seen * hkv * 2 * d * es + io + 4 * (seen // PAGE + 3 * len(ln)), "flops": 4 * d * hq * rows}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _cache(nb, case, scale, gen):
    """A cache of rows of unit variance: bf16, or uint8 e4m3fn codes."""
    shape = (nb, PAGE, case["hkv"], case["d"])
    c = torch.empty(shape, dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (PAGE * case["hkv"] * case["d"]))
    for a in range(0, nb, step):
        x = torch.randn(min(step, nb - a), *shape[1:], generator=gen, device="cuda")
        c[a:a + step] = x.to(torch.bfloat16) if case["kv"] == "bf16" else \
            (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    return c


def _positions(case, r):
    """int32 [axes, T]: text, whose axes advance together, and images, whose height and width vary within."""
    t, a = case["tokens"], case["axes"]
    pos = np.zeros((a, t), dtype=np.int64)
    at, here = 0, int(r.integers(0, 20000))
    while at < t:
        n = min(t - at, int(r.integers(1, 400)))
        if a > 1 and r.random() < 0.5:                    # an image of n patches, in rows of w
            w = int(r.integers(1, 33))
            k = np.arange(n)
            for x in range(a):
                pos[x, at:at + n] = here + (0 if x == 0 else k // w if x == 1 else k % w)
            here += max(w, n // w + 1)
        else:
            pos[:, at:at + n] = here + np.arange(n)
            here += n
        at += n
    return pos, here + 1


def prepare(case, seed):
    op, gen, r = case["op"], _gen(seed), np.random.default_rng(seed)
    st = {"op": op, "case": case}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "rope":
        t, nb = case["tokens"], case["pool"]
        for name, h in (("query", hq), ("key", hkv), ("value", hkv)):
            st[name] = torch.randn(t, h, d, generator=gen, device="cuda").to(torch.bfloat16)
        pos, n = _positions(case, r)
        st["pos"] = _i32(pos)
        # the program's table: cosines, then sines, of every position's angles
        angle = np.arange(n, dtype=np.float64)[:, None] * \
            THETA ** (-2.0 * np.arange(case["rot"] // 2, dtype=np.float64) / case["rot"])[None]
        st["table"] = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
        st["axis"] = _pair_axis(case)
        st["axis_t"] = torch.tensor(st["axis"], device="cuda")
        slots = r.permutation(nb * PAGE)[:t]
        slots[r.random(t) < 0.02] = -1                    # padding tokens
        st["slots"] = _i32(slots)
        st["k"], st["v"] = _cache(nb, case, K_SCALE, gen), _cache(nb, case, V_SCALE, gen)
        st["out"] = torch.empty_like(st["query"])
        return st
    ln, qn = _lens(case)
    own_pages, shared, width = -(-ln // PAGE), None, None
    if op == "shared":
        at, pre = _groups(case)
        of = np.repeat(np.arange(case["groups"]), np.diff(at))
        whole = pre // PAGE                               # pages in common; the rest of a page is each sequence's own
        ln = ln + pre[of]
        own_pages = -(-ln // PAGE) - whole[of]
        st["group_at"], st["whole"] = at.tolist(), whole.tolist()
        st["gsl"], st["shared"] = _i32(at), _i32(pre)
        st["of"] = torch.from_numpy(of).cuda()
        shared = whole
    total = int(own_pages.sum() + (shared.sum() if shared is not None else 0))
    nb = int(math.ceil(1.1 * total))
    ids = r.permutation(nb)
    width = int((-(-ln // PAGE)).max())
    bt, at_id = np.full((len(ln), width), -1, dtype=np.int64), 0
    heads = []
    if shared is not None:
        for w in shared:
            heads.append(ids[at_id:at_id + w])
            at_id += w
    for i, n in enumerate(own_pages):
        h = 0
        if shared is not None:
            h = len(heads[of[i]])
            bt[i, :h] = heads[of[i]]
        bt[i, h:h + n] = ids[at_id:at_id + n]
        at_id += n
    st["k"], st["v"] = _cache(nb, case, K_SCALE, gen), _cache(nb, case, V_SCALE, gen)
    st["bt"], st["sl"] = _i32(bt), _i32(ln)
    st["qsl"] = _i32(np.concatenate([[0], np.cumsum(qn)])) if case["runs"] > 1 else None
    st["len"], st["qn"] = torch.from_numpy(ln).cuda(), torch.from_numpy(qn).cuda()
    st["longest"], st["own_longest"] = int(ln.max()), int(own_pages.max()) * PAGE
    t = int(qn.sum())
    # where each query token stands in a batch padded to the longest run
    seq = np.repeat(np.arange(len(qn)), qn)
    st["seq"] = torch.from_numpy(seq).cuda()
    st["row"] = torch.from_numpy(np.arange(t) - (np.cumsum(qn) - qn)[seq]).cuda()
    st["q"] = torch.randn(t, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(t, hq, device="cuda")
    if own:
        from paged_kv_decode_06_gb300 import binding
        args = (st["q"], st["k"], st["v"], st["bt"], st["sl"], st["qsl"], case["runs"])
        rest = {"scale": d ** -0.5, "k_scale": K_SCALE, "v_scale": V_SCALE, "out": st["out"], "lse": st["lse"]}
        if op == "window":
            st["call"] = binding.prepare_decode_window(*args, case["window"], case["first"], **rest)
        else:
            st["call"] = binding.prepare_decode_shared(*args, st["gsl"], st["shared"], **rest)
    return st


# ---------------------------------------------------------------- plain forms

def _real(rows, case, scale):
    """Cached rows as float32 values."""
    return rows.float() if case["kv"] == "bf16" else rows.view(torch.float8_e4m3fn).float() * scale


def _rotated(x, cos, sin, case):
    """float32 rows [T, H, D], their first `rot` features rotated pair by pair."""
    n = case["rot"] // 2
    if case["pairs"] == "halves":
        a, b = x[..., :n], x[..., n:2 * n]
        parts = [a * cos - b * sin, b * cos + a * sin]
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        parts = [torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)]
    return torch.cat(parts + [x[..., 2 * n:]], -1)


def _plain_rope(st):
    c = st["case"]
    n = c["rot"] // 2
    pos = st["pos"].long()[st["axis_t"]]                            # [pairs, T]
    col = torch.arange(n, device=pos.device).unsqueeze(1)
    cos, sin = st["table"][pos, col].t().unsqueeze(1), st["table"][pos, n + col].t().unsqueeze(1)
    st["out"].copy_(_rotated(st["query"].float(), cos, sin, c).to(torch.bfloat16))
    slots = st["slots"].long()
    live = (slots >= 0).nonzero().squeeze(1)
    page, off = slots[live] // PAGE, slots[live] % PAGE
    for x, cache, scale in ((_rotated(st["key"].float(), cos, sin, c), st["k"], K_SCALE),
                            (st["value"].float(), st["v"], V_SCALE)):
        if c["kv"] == "bf16":
            cache[page, off] = x[live].to(torch.bfloat16)
        else:
            q = x[live] / torch.full((), scale, device=x.device)
            cache[page, off] = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _part(st, q, tok, seen):
    """Attention of padded query rows over some cached tokens: the largest score, the sum of the weights
    beside it and the weighted values.  q [N, R, Hq, D]; tok (page, slot) [N, K]; seen [N, R, K]."""
    c = st["case"]
    n, rr = q.shape[:2]
    hkv, d = c["hkv"], c["d"]
    g = c["hq"] // hkv
    k = _real(st["k"][tok], c, K_SCALE).permute(0, 2, 3, 1)          # [N, Hkv, D, K]
    qh = q.reshape(n, rr, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, rr * g, d)
    s = torch.matmul(qh, k) * d ** -0.5
    if seen is not None:
        s.masked_fill_(~seen.repeat_interleave(g, 1).unsqueeze(1), -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    o = torch.matmul(e, _real(st["v"][tok], c, V_SCALE).transpose(1, 2))

    def back(x):                                                     # [N, Hkv, R * G, X] -> [N, R, Hq, X]
        return x.reshape(n, hkv, rr, g, -1).permute(0, 2, 1, 3, 4).reshape(n, rr, c["hq"], -1)
    return back(m), back(e.sum(-1, keepdim=True)), back(o)


def _padded(st):
    """Query rows padded to the longest run, and their positions."""
    c = st["case"]
    q = torch.zeros(c["batch"], c["runs"], c["hq"], c["d"], device="cuda")
    q[st["seq"], st["row"]] = st["q"].float()
    pos = (st["len"] - st["qn"]).unsqueeze(1) + torch.arange(c["runs"], device="cuda")
    return q, pos


def _finish(st, m, z, o):
    st["out"].copy_((o / z).to(torch.bfloat16))
    st["lse"].copy_((m + torch.log(z)).squeeze(-1))
    return st["out"], st["lse"]


def _where(st, j):
    """(page, slot) of logical tokens j [N, K]; those past a table row's end take its first entry's."""
    page = torch.gather(st["bt"].long(), 1, (j // PAGE).clamp(max=st["bt"].shape[1] - 1))
    return page.clamp(min=0), j % PAGE


def _plain_window(st):
    c = st["case"]
    q, pos = _padded(st)
    w, f = c["window"], min(c["first"], st["longest"])
    start = (st["len"] - st["qn"] - w + 1).clamp(min=f).unsqueeze(1)
    near = start + torch.arange(min(w + c["runs"] - 1, st["longest"]), device="cuda")
    j = torch.cat([torch.arange(f, device="cuda").expand(c["batch"], f), near], 1)
    jj, p = j.unsqueeze(1), pos.unsqueeze(2)
    m, z, o = _part(st, q, _where(st, j), (jj <= p) & ((jj > p - w) | (jj < f)))
    at = (st["seq"], st["row"])
    return _finish(st, m[at], z[at], o[at])


def _plain_shared(st):
    c = st["case"]
    q, pos = _padded(st)
    # each sequence's own tokens, behind the pages in common
    skip = torch.tensor(st["whole"], device="cuda")[st["of"]].unsqueeze(1) * PAGE
    j = skip + torch.arange(st["own_longest"], device="cuda")
    m, z, o = _part(st, q, _where(st, j), j.unsqueeze(1) <= pos.unsqueeze(2))
    # the pages in common, once for a group's rows
    for a, b, w in zip(st["group_at"], st["group_at"][1:], st["whole"]):
        if w == 0:
            continue
        tok = (st["bt"][a, :w].long().repeat_interleave(PAGE).unsqueeze(0),
               torch.arange(PAGE, device="cuda").repeat(w).unsqueeze(0))
        pm, pz, po = _part(st, q[a:b].reshape(1, -1, c["hq"], c["d"]), tok, None)
        pm, pz, po = (x.reshape(b - a, c["runs"], c["hq"], -1) for x in (pm, pz, po))
        top = torch.maximum(m[a:b], pm)
        x, y = torch.exp(m[a:b] - top), torch.exp(pm - top)
        m[a:b], z[a:b], o[a:b] = top, z[a:b] * x + pz * y, o[a:b] * x + po * y
    at = (st["seq"], st["row"])
    return _finish(st, m[at], z[at], o[at])


# ------------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if op == "rope":
        if own:
            from paged_kv_decode_06_gb300 import binding
            c = st["case"]
            binding.paged_attn_rope_cache_write(
                st["query"], st["key"], st["value"], st["pos"], st["table"], st["slots"], st["k"], st["v"],
                pair_axis=st["axis"], neighbours=c["pairs"] == "neighbours", k_scale=K_SCALE, v_scale=V_SCALE,
                query_out=st["out"])
        else:
            _plain_rope(st)
        if st["case"]["kv"] == "fp8":
            return st["out"], st["k"].view(torch.float8_e4m3fn), st["v"].view(torch.float8_e4m3fn)
        return st["out"], st["k"], st["v"]
    if own:
        return st["call"]()
    return _plain_window(st) if op == "window" else _plain_shared(st)


# -------------------------------------------------- the definitions in 64 bits

def _nearest_e4m3(x):
    """The nearest finite e4m3fn value (ties to the even code, 448 beyond): three bits of mantissa, bias 7, subnormals
    in steps of 2^-9."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_rope(case, st):
    t, n = case["tokens"], case["rot"] // 2
    pos, table = st["pos"].cpu().numpy(), st["table"].double()

    def rotate(x):
        y = x.double().clone()
        for i, a in enumerate(st["axis"]):
            u, v = (i, i + n) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
            p = torch.from_numpy(pos[a].astype(np.int64)).cuda()
            co, si = table[p, i].reshape(t, 1), table[p, n + i].reshape(t, 1)
            y[:, :, u] = x[:, :, u].double() * co - x[:, :, v].double() * si
            y[:, :, v] = x[:, :, v].double() * co + x[:, :, u].double() * si
        return y

    slots = st["slots"].long()
    live = slots >= 0
    res = [rotate(st["query"])]
    for cache, rows, scale in ((st["k"], rotate(st["key"]), K_SCALE), (st["v"], st["value"].double(), V_SCALE)):
        if case["kv"] == "fp8":
            whole, rows = cache.view(torch.float8_e4m3fn).double(), _nearest_e4m3(rows / float(np.float32(scale)))
        else:
            whole = cache.double()
        flat = whole.reshape(-1, case["hkv"], case["d"]).clone()
        flat[slots[live]] = rows[live]
        res.append(flat.reshape(whole.shape))
    return res


def _exact_attention(case, st):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, t = hq // hkv, 0
    ks, vs = (float(np.float32(s)) if case["kv"] == "fp8" else 1.0 for s in (K_SCALE, V_SCALE))
    real = (lambda x: x.double()) if case["kv"] == "bf16" else (lambda x: x.view(torch.float8_e4m3fn).double())
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (l, qn) in enumerate(zip(st["len"].tolist(), st["qn"].tolist())):
        j = torch.arange(l, device="cuda")
        if case["op"] == "window":                        # what no row of the sequence sees is left out
            j = j[(j < case["first"]) | (j > l - qn - case["window"])]
        page, off = st["bt"][i].long()[j // PAGE], j % PAGE
        k, v = real(st["k"][page, off]) * ks, real(st["v"][page, off]) * vs
        for r in range(qn):
            p = l - qn + r
            keep = j <= p
            if case["op"] == "window":
                keep &= (j > p - case["window"]) | (j < case["first"])
            s = torch.einsum("hgd,jhd->hgj", st["q"][t].double().reshape(hkv, g, d), k) / math.sqrt(d)
            s = s.masked_fill(~keep, -math.inf)
            z = torch.logsumexp(s, -1)
            out[t] = torch.einsum("hgj,jhd->hgd", torch.exp(s - z.unsqueeze(-1)), v).reshape(hq, d)
            lse[t] = z.reshape(hq)
            t += 1
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rope(case, st) if case["op"] == "rope" else _exact_attention(case, st)
