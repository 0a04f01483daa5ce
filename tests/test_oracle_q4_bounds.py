"""The bounds of oracle.cache_q4.decode_with_bounds on the CPU: an evaluation with
the kernel's roundings stays inside them, planted mistakes do not."""
import numpy as np
import pytest

from oracle import cache_q4


def needle_case(L, d, hq, hkv, seed, sinks=None, window=0, gain=2.0):
    """One sequence of L tokens, one query row a head, each row along the key of a token of its own: that
    token has nearly all of the row's weight, so what its page holds decides the row.  The other scores
    have a standard deviation of `gain`."""
    r = np.random.default_rng(seed)
    nb = -(-L // 16) + 2
    bt = r.permutation(nb)[None, :nb - 2].astype(np.int32)
    codes = [r.integers(0, 256, (nb, 16, hkv, d // 2)).astype(np.uint8) for _ in range(2)]
    scales = [r.integers(0x28, 0x38, (nb, hkv, 16, d // 16)).astype(np.uint8) for _ in range(2)]
    first = max(0, L - window) if window else 0
    at = first + r.permutation(L - first)[:hq]
    k = cache_q4.dequantise_rows(codes[0], scales[0].transpose(0, 2, 1, 3), 0.02)
    q = np.stack([k[bt[0, a // 16], a % 16, h // (hq // hkv)] for h, a in enumerate(at)])
    q = q * gain / (np.sqrt((q ** 2).sum(-1, keepdims=True)) * k.std())
    q = np.float32(q).view(np.uint32) & 0xFFFF0000          # bf16 values
    q = q.view(np.float32).astype(np.float64)[None]
    return dict(q=q, codes=codes, scales=scales, bt=bt, lens=np.array([L], dtype=np.int32), sinks=sinks, at=at,
                scale=1.0, window=window)


def bounds(c, codes=None):
    return cache_q4.decode_with_bounds(c["q"], codes or c["codes"], c["scales"], c["bt"], c["lens"], None, c["scale"],
                                       0.02, 0.03, c["window"], c["sinks"])


def rounded(c, maximum=None):
    """The row outputs in float64 but for weights rounded to f16 below `maximum` (default: the keys' own)."""
    L = int(c["lens"][0])
    j = np.arange(max(0, L - c["window"]) if c["window"] else 0, L)
    page, off = c["bt"][0][j // 16], j % 16
    k = cache_q4.dequantise_rows(c["codes"][0][page, off], c["scales"][0][page, :, off], 0.02)
    v = cache_q4.dequantise_rows(c["codes"][1][page, off], c["scales"][1][page, :, off], 0.03)
    out = np.empty_like(c["q"])
    g = out.shape[1] // k.shape[1]
    for h in range(out.shape[1]):
        s = c["scale"] * (k[:, h // g] @ c["q"][0, h])
        m = s.max() if maximum is None else max(s.max(), maximum[h])
        p = np.exp(s - m)
        total = p.sum() + (np.exp(c["sinks"][h] - m) if c["sinks"] is not None else 0.0)
        out[0, h] = p.astype(np.float16).astype(np.float64) @ v[:, h // g] / total
    return out


def _outside(got, want, tol):
    return bool((np.abs(got - want) > tol).any())


@pytest.mark.parametrize("L,d,hq,hkv,window", [(20000, 64, 16, 1, 0), (3000, 128, 8, 2, 500)])
def test_planted_mistakes_are_outside_the_bounds(L, d, hq, hkv, window):
    c = needle_case(L, d, hq, hkv, seed=L, window=window)
    out, lse, tol, _ = bounds(c)
    assert not _outside(rounded(c), out, tol)
    assert _outside(np.zeros_like(out), out, tol)
    for a in c["at"][:4]:                                    # one page's values lost
        v = c["codes"][1].copy()
        v[c["bt"][0, a // 16]] = 0
        assert _outside(bounds(c, [c["codes"][0], v])[0], out, tol)
    assert _outside(np.roll(out, 1, axis=1), out, tol)       # heads exchanged


def test_even_weights_too():
    """All keys alike in weight: the output is a mean far below the values, and still bounded by them."""
    c = needle_case(20000, 64, 4, 1, seed=1, gain=0.3)
    out, _, tol, _ = bounds(c)
    assert not _outside(rounded(c), out, tol) and _outside(np.zeros_like(out), out, tol)
    v = c["codes"][1].copy()
    v[c["bt"][0, :200]] = 0
    assert _outside(bounds(c, [c["codes"][0], v])[0], out, tol)


@pytest.mark.parametrize("above", [17.0, 20.0, 25.0])
def test_weights_rounded_against_the_sink_are_outside(above):
    c = needle_case(512, 128, 4, 1, seed=2, gain=0.5)
    c["sinks"] = np.full(4, above, dtype=np.float32)         # the mean score is 0
    out, _, tol, _ = bounds(c)
    assert not _outside(rounded(c), out, tol)
    assert _outside(rounded(c, maximum=c["sinks"]), out, tol)
