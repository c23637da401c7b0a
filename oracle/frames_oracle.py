"""Oracle of the windowed attention and the 8-bit cache: plain fp64 numpy, one
row at a time, and a model of the page bookkeeping. Test infrastructure only;
the product path never imports it.
"""
from __future__ import annotations

import numpy as np

LOG2_MIN_SCALE = -110
E4M3_MAX = 448.0


# ---- visibility and attention ----------------------------------------------
def visible(p, L, frame=1, window=0, sinks=0, causal=1):
    """Truth for every key j < L: seen from position p."""
    j = np.arange(L)
    if p < 0:
        return np.zeros(L, bool)
    fq, fj = p // frame, j // frame
    see = np.ones(L, bool)
    if causal:
        see &= fj <= fq
    if window:
        see &= (np.abs(fq - fj) < window) | (fj < sinks)
    return see


def attention(q, k, v, n, see, scale=0.0):
    """q [Hq, Nq, d], k and v [Hkv, L, d] of one sequence, its first n query
    rows: (out, lse, weight) in fp64 plus, per row, `spread`: scale * max_j
    sum_c |q_c k_jc| over visible keys, and `mass` [.., d]: sum_j p_j |v_j|,
    from which tests derive their tolerances. Rows that see nothing: 0, -inf."""
    Hq, _, d = q.shape
    group = Hq // k.shape[0]
    L = k.shape[1]
    scale = scale or d ** -0.5
    out, mass = np.zeros((Hq, n, d)), np.zeros((Hq, n, d))
    lse, spread = np.full((Hq, n), -np.inf), np.zeros((Hq, n))
    for i in range(n):
        on = np.flatnonzero(visible(L - n + i, L, **see))
        if on.size == 0:
            continue
        for h in range(Hq):
            kk, vv = k[h // group, on], v[h // group, on]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (kk @ q[h, i])
                m = s.max()
                e = np.exp(s - m)
                out[h, i] = (e / e.sum()) @ vv
                mass[h, i] = (e / e.sum()) @ np.abs(vv)
                lse[h, i] = m + np.log(e.sum())
                spread[h, i] = scale * (np.abs(kk) @ np.abs(q[h, i])).max()
    return dict(out=out, lse=lse, mass=mass, spread=spread)


# ---- e4m3 -------------------------------------------------------------------
def e4m3_table():
    """The value of each of the 256 codes (0x7f and 0xff: NaN)."""
    c = np.arange(256)
    s, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, c & 7
    x = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    x = s * x
    x[[0x7F, 0xFF]] = np.nan
    return x


TABLE = e4m3_table()
_POS = TABLE[:0x7F]  # ascending, 0 .. 448


def e4m3_encode(x):
    """Codes of the nearest e4m3 values, ties to the even code; NaN and values
    that are not finite become NaN (0x7f)."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= E4M3_MAX, 0x7E, code)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_for(amax):
    """The smallest power of two s >= 2^-110 with amax <= 448 s."""
    s = 2.0 ** LOG2_MIN_SCALE
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


# ---- the cache ----------------------------------------------------------------
class CacheModel:
    """Host model of a paged cache: codes, scales, table, lengths, counts."""

    def __init__(self, p):
        self.p = dict(p)
        shape = (p["n_pages"], p["Hkv"], p["page"], p["d"])
        self.k8, self.v8 = np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)
        self.k_scale, self.v_scale = np.ones(shape[:2]), np.ones(shape[:2])
        self.table = np.full((p["B"], p["max_pages"]), -1, np.int64)
        self.len = np.zeros(p["B"], np.int64)
        self.ref = np.zeros(p["n_pages"], np.int64)

    def reserve(self, n_new):
        """Lengths before, or None when nothing was done."""
        p, page = self.p, self.p["page"]
        if any(n < 0 for n in n_new):
            return None
        free = [int(x) for x in np.flatnonzero(self.ref == 0)]
        want, plan = 0, []
        for b, n in enumerate(n_new):
            L = int(self.len[b])
            if L + n > p["max_pages"] * page:
                return None
            have, need = -(-L // page), -(-(L + n) // page)
            copy = bool(n and L % page and self.ref[self.table[b, L // page]] > 1)
            plan.append((have, need, copy))
            want += need - have + copy
        if want > len(free):
            return None
        old = [int(self.table[b, self.len[b] // page]) if c else -1
               for b, (_, _, c) in enumerate(plan)]
        for b, (have, need, copy) in enumerate(plan):
            cols = ([have - 1] if copy else []) + list(range(have, need))
            for col in cols:
                x = free.pop(0)
                if copy and col == have - 1:
                    for t in (self.k8, self.v8, self.k_scale, self.v_scale):
                        t[x] = t[old[b]]
                    self.ref[old[b]] -= 1
                self.table[b, col] = x
                self.ref[x] = 1
        start = self.len.copy()
        self.len += np.asarray(n_new)
        return start

    def append(self, k, v, start, n_new):
        """k, v [B, Hkv, T, d] in fp64."""
        page = self.p["page"]
        for x, x8, scale in ((k, self.k8, self.k_scale), (v, self.v8, self.v_scale)):
            for b in range(self.p["B"]):
                lo, end = int(start[b]), int(start[b]) + int(n_new[b])
                if lo < 0:
                    continue
                for col in range(lo // page, -(-end // page)):
                    pg = self.table[b, col]
                    t0, t1 = max(lo, col * page), min(end, (col + 1) * page)
                    held = t0 - col * page
                    for h in range(self.p["Hkv"]):
                        new = x[b, h, t0 - lo:t1 - lo]
                        fin = np.abs(new[np.isfinite(new)])
                        s = scale_for(fin.max() if fin.size else 0.0)
                        if held:
                            s = max(s, scale[pg, h])
                            if s != scale[pg, h]:
                                old = TABLE[x8[pg, h, :held]] * (scale[pg, h] / s)
                                x8[pg, h, :held] = e4m3_encode(old)
                        x8[pg, h, held:t1 - col * page] = e4m3_encode(new / s)
                        scale[pg, h] = s

    def tokens(self, b, which="k"):
        """The tokens of sequence b as the cache stands for them: [Hkv, L, d]
        (NaN where a page is missing)."""
        x8, scale = (self.k8, self.k_scale) if which == "k" else (self.v8, self.v_scale)
        L, page = int(self.len[b]), self.p["page"]
        out = np.full((self.p["Hkv"], L, self.p["d"]), np.nan)
        for t in range(0, L, page):
            pg = self.table[b, t // page]
            if pg >= 0:
                n = min(page, L - t)
                out[:, t:t + n] = TABLE[x8[pg, :, :n]] * scale[pg][:, None, None]
        return out

    def fork(self, src, dst):
        src, dst = list(src), list(dst)
        B = self.p["B"]
        good = [0 <= s < B and 0 <= t < B and self.len[t] == 0 and dst.count(t) == 1
                and t not in src for s, t in zip(src, dst)]
        for (s, t), ok in zip(zip(src, dst), good):
            if ok:
                self.table[t] = self.table[s]
                self.len[t] = self.len[s]
                for x in self.table[s][self.table[s] >= 0]:
                    self.ref[x] += 1
        return all(good)

    def _give_up(self, b, cols):
        for c in cols:
            if self.table[b, c] >= 0:
                self.ref[self.table[b, c]] -= 1
                self.table[b, c] = -1

    def free(self, seqs):
        for b in set(int(s) for s in seqs):
            if 0 <= b < self.p["B"]:
                self._give_up(b, range(self.p["max_pages"]))
                self.len[b] = 0

    def evict(self, frame, window, sinks):
        page = self.p["page"]
        for b in range(self.p["B"]):
            L = int(self.len[b])
            seen = visible(L, L + 1, frame, window, sinks, 1)
            for c in range(L // page):
                if not seen[c * page:(c + 1) * page].any():
                    self._give_up(b, [c])

    def compact(self):
        used = int((self.ref > 0).sum())
        src = [x for x in range(used, self.p["n_pages"]) if self.ref[x] > 0]
        dst = [x for x in range(used) if self.ref[x] == 0]
        for s, t in zip(src, dst):
            for a in (self.k8, self.v8, self.k_scale, self.v_scale):
                a[t] = a[s]
            self.table[self.table == s] = t
            self.ref[t], self.ref[s] = self.ref[s], 0
        return used
