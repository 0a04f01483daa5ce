"""Plain CPU statement of the page operations (TEST INFRASTRUCTURE ONLY), entry
by entry as include/paged_attn.h defines them.  Arrays are NumPy and updated in
place; every function returns the bits the device status word would gain."""
from __future__ import annotations

import numpy as np

PAGE = 16
BAD_PAGE, BAD_LEN, REFUSED = 1, 2, 32


def copy(caches, src, dst):
    st, nb = 0, caches[0].shape[0]
    old = [c.copy() for c in caches]
    for s, d in zip(src, dst):
        if s < 0 or d < 0:
            continue
        if s >= nb or d >= nb:
            st |= BAD_PAGE
            continue
        for c, o in zip(caches, old):
            c[d] = o[s]
    return st


def fork(caches, bt, sl, ref, parents, children, new):
    st, nb = 0, len(ref)
    sl0, ref0, new0 = sl.copy(), ref.copy(), new.copy()
    live = [k for k in range(len(parents)) if parents[k] >= 0 and children[k] >= 0]
    new[:] = -1
    for k in live:
        p, c = parents[k], children[k]
        ok = p < len(sl) and c < len(sl) and sl0[p] >= 0 and sl0[c] == 0
        if ok:
            full, rest = divmod(int(sl0[p]), PAGE)
            ok = full + (rest > 0) <= bt.shape[1]
            ok = ok and not any(parents[x] == c for x in live)
            ok = ok and not any(children[x] == c for x in live if x < k)
            if rest:
                ok = ok and 0 <= new0[k] < nb and ref0[new0[k]] == 0
                ok = ok and not any(new0[x] == new0[k] for x in live if x < k)
        if not ok:
            st |= REFUSED
            continue
        for j in range(full):
            bt[c, j] = bt[p, j]
            if 0 <= bt[p, j] < nb:
                ref[bt[p, j]] += 1
            else:
                st |= BAD_PAGE
        if rest:
            new[k] = bt[c, full] = new0[k]
            ref[new0[k]] = 1
            if 0 <= bt[p, full] < nb:
                for x in caches:
                    x[new0[k]] = x[bt[p, full]]
            else:
                st |= BAD_PAGE
        sl[c] = sl0[p]
    return st


def free(bt, sl, ref, rows):
    st, nb = 0, len(ref)
    for r in rows:
        if r < 0:
            continue
        if r >= len(sl):
            st |= REFUSED
            continue
        held = -(-int(max(sl[r], 0)) // PAGE)
        sl[r] = 0
        if held > bt.shape[1]:
            st |= BAD_LEN
            held = bt.shape[1]
        for p in bt[r, :held]:
            if not 0 <= p < nb:
                st |= BAD_PAGE
            elif ref[p] <= 0:
                st |= REFUSED
            else:
                ref[p] -= 1
    ids = np.flatnonzero(ref <= 0)
    out = np.full(nb, -1, dtype=np.int32)
    out[:len(ids)] = ids
    return st, out, len(ids)


def compact(caches, bt, ref):
    st = REFUSED if (ref < 0).any() else 0
    nb = len(ref)
    used = ref > 0
    n = int(used.sum())
    page_map = np.where(used, np.arange(nb), -1).astype(np.int32)
    high = [p for p in range(n, nb) if used[p]]
    holes = [p for p in range(n) if not used[p]]
    ref[ref < 0] = 0
    for src, dst in zip(high, holes):
        for c in caches:
            c[dst] = c[src]
        page_map[src] = dst
        ref[dst], ref[src] = ref[src], 0
    for idx in np.ndindex(bt.shape):
        if 0 <= bt[idx] < nb and page_map[bt[idx]] >= 0:
            bt[idx] = page_map[bt[idx]]
    return st, page_map, n
