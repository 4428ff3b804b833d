"""Head norm and rotation, the paged E4M3 key/value cache, attention over it, in
64 bits.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definitions (token by token, from the formulas in include/fp8sm.h):
  norm_rope   y = x / sqrt(mean(x^2) + eps) * w, then each pair (a, b) of the
              first `rot` values becomes (a c - b s, b c + a s)
  write       per touched block, head, K or V: e = the smallest integer with
              448 * 2^e >= max(max|new|, 1e-10) (finite values only), not below
              the exponent of a block that holds tokens; code = E4M3(x 2^-e),
              held codes re-encoded when the exponent rises
  values      code * 2^(byte - 127)
  attention   softmax over the visible tokens, written as plain sums

Pins (tests/test_oracle_kv.py): rotations keep lengths and compose; a write of
one fresh block equals the pinned UE8M0 group quant of the block as one group;
a token-by-token write equals the closed form of each block's final exponent;
attention equals torch's float64 softmax on dense copies and closed forms.
"""
import numpy as np

from . import e4m3


def norm_rope(x, Hq, Hk, D, pos=None, cos_sin=None, wq=None, wk=None, eps=1e-6, interleaved=False):
    """x [T, >= (Hq + Hk) D] -> (y float64 [T, Hq + Hk, D], magnitude of each
    output's summands).  Rows at positions outside the table: NaN."""
    T = x.shape[0]
    y = np.asarray(x, dtype=np.float64)[:, :(Hq + Hk) * D].reshape(T, Hq + Hk, D).copy()
    if wq is not None:
        y /= np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        y[:, :Hq] *= np.asarray(wq, dtype=np.float64)
        y[:, Hq:] *= np.asarray(wk, dtype=np.float64)
    mag = np.abs(y)
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        half = rot // 2
        first = np.arange(half) * (2 if interleaved else 1)
        second = first + (1 if interleaved else half)
        for t in range(T):
            if not 0 <= pos[t] < cos_sin.shape[0]:
                y[t] = np.nan
                continue
            c, s = cos_sin[pos[t], :half].astype(np.float64), cos_sin[pos[t], half:].astype(np.float64)
            a, b = y[t][:, first].copy(), y[t][:, second].copy()
            y[t][:, first] = a * c - b * s
            y[t][:, second] = b * c + a * s
            mag[t][:, first] = np.abs(a * c) + np.abs(b * s)
            mag[t][:, second] = np.abs(b * c) + np.abs(a * s)
    return y, mag


class Cache:
    """The four arrays of a cache (see include/fp8sm.h), as numpy uint8."""

    def __init__(self, k, v, ke, ve):
        self.codes = [np.array(k), np.array(v)]
        self.exp = [np.array(ke), np.array(ve)]
        self.blocks, self.H, self.block, self.D = self.codes[0].shape

    def get(self, which, page, slot, h):
        c = self.codes[which]
        return c[page, h, slot] if which == 0 else c[page, h, slot // 16, :, slot % 16]

    def put(self, which, page, slot, h, codes):
        if which == 0:
            self.codes[0][page, h, slot] = codes
        else:
            self.codes[1][page, h, slot // 16, :, slot % 16] = codes

    def token(self, which, page, slot):
        """Values [H, D] of one token."""
        return np.stack([e4m3.decode(self.get(which, page, slot, h)) * 2.0 ** (int(self.exp[which][page, h]) - 127)
                         for h in range(self.H)])


def rows_of(cu, lens, b, T, reach):
    """(first row, new tokens, cached length) of sequence b, clamped."""
    c0 = min(max(int(cu[b]), 0), T)
    n = min(max(int(cu[b + 1]), c0), T) - c0
    return c0, n, min(max(int(lens[b]), 0), reach)


def exponent(amax):
    a = max(float(amax), float(np.float32(1e-10)))
    m, e = np.frexp(a / 448.0)
    return int(e) - 1 if m == 0.5 else int(e)


def _encode(x):
    nan = np.isnan(x)
    c = e4m3.encode(np.clip(np.where(nan, 0.0, x), -448, 448).astype(np.float64))
    return np.where(nan, 0x7F, c).astype(np.uint8)


def write(cache, k, v, cu, lens, table):
    """k, v [T, H, D]; changes `cache`."""
    T, block = k.shape[0], cache.block
    for b in range(len(lens)):
        c0, n, L = rows_of(cu, lens, b, T, table.shape[1] * block)
        start = L - n
        for j in range(max(start, 0) // block, -(-L // block)):
            lo, hi = max(start, j * block, 0), min(L, (j + 1) * block)
            page = int(table[b, j])
            if hi <= lo or not 0 <= page < cache.blocks:
                continue
            held = lo - j * block
            for which, x in ((0, k), (1, v)):
                for h in range(cache.H):
                    new = np.asarray(x[c0 + lo - start:c0 + hi - start, h], dtype=np.float64)
                    fin = np.abs(new[np.isfinite(new)])
                    e = exponent(fin.max() if fin.size else 0.0)
                    if held:
                        old = int(cache.exp[which][page, h]) - 127
                        if e > old:
                            for s in range(held):
                                c = cache.get(which, page, s, h)
                                cache.put(which, page, s, h, _encode(e4m3.decode(c) * 2.0 ** (old - e)))
                        e = max(e, old)
                    cache.exp[which][page, h] = e + 127
                    for s in range(lo, hi):
                        cache.put(which, page, s - j * block, h, _encode(new[s - lo] * 2.0 ** -e))


def read(cache, cu, lens, table, total):
    """-> (k, v) float64 [total, H, D]; rows of no sequence NaN."""
    out = []
    for which in (0, 1):
        x = np.full((total, cache.H, cache.D), np.nan)
        for b in range(len(lens)):
            c0, n, L = rows_of(cu, lens, b, total, table.shape[1] * cache.block)
            for i in range(n):
                p = L - n + i
                page = int(table[b, p // cache.block]) if p >= 0 else -1
                x[c0 + i] = cache.token(which, page, p % cache.block) if 0 <= page < cache.blocks else 0.0
        out.append(x)
    return out


def attention(q, cache, cu, lens, table, scale, causal=True, window=0):
    """q [T, Hq, D] -> (out, lse, spread, qk): float64 [T, Hq, D], [T, Hq], the
    probability-weighted |v| of every output and the largest sum |q||k| of every
    row (for error bounds).  Rows of no sequence: NaN."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    spread = np.zeros((T, Hq, D))
    qk = np.zeros((T, Hq))
    q = np.asarray(q, dtype=np.float64)
    for b in range(len(lens)):
        c0, n, L = rows_of(cu, lens, b, T, table.shape[1] * cache.block)
        if n == 0:
            continue
        pages = [int(table[b, p // cache.block]) for p in range(L)]
        there = np.array([0 <= g < cache.blocks for g in pages], dtype=bool)
        keys = np.zeros((L, cache.H, D))
        vals = np.zeros((L, cache.H, D))
        for p in np.nonzero(there)[0]:
            keys[p] = cache.token(0, pages[p], p % cache.block)
            vals[p] = cache.token(1, pages[p], p % cache.block)
        for i in range(n):
            pos = L - n + i
            hi = min(L, pos + 1) if causal else L
            lo = max(pos - window + 1, 0) if window else 0
            seen = np.nonzero(there[lo:max(hi, lo)])[0] + lo
            for h in range(Hq):
                if len(seen) == 0:
                    out[c0 + i, h], lse[c0 + i, h] = 0.0, -np.inf
                    continue
                kh, vh = keys[seen, h // G], vals[seen, h // G]
                s = kh @ q[c0 + i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                out[c0 + i, h] = p @ vh / p.sum()
                spread[c0 + i, h] = p @ np.abs(vh) / p.sum()
                lse[c0 + i, h] = m + np.log(p.sum())
                qk[c0 + i, h] = (np.abs(kh) @ np.abs(q[c0 + i, h])).max()
    return out, lse, spread, qk
