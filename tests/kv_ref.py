"""The key/value cache calls written out plainly on the host, in float64 and in the order of
specverify.h: what the GPU tests compare with."""
import math

import numpy as np

MIN_EXP = -64
XMAX = 448.0 * 2.0 ** 64


def e4m3(x):
    """Nearest e4m3 value, ties to even, saturating at 448 (NaN stays)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def scale_for(a):
    """Smallest 2^e >= a / 448, e >= MIN_EXP."""
    e = MIN_EXP
    while 448.0 * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


class RefCache:
    def __init__(self, layers, pages, page, heads, dim, batch, max_pages):
        self.layers, self.pages, self.page, self.heads = layers, pages, page, heads
        self.dim, self.batch, self.max_pages = dim, batch, max_pages
        # [kv][layer, page, head, slot, dim] e4m3 values and [kv][layer, page, head] scales
        self.q = np.zeros((2, layers, pages, heads, page, dim))
        self.s = np.ones((2, layers, pages, heads))
        self.rows = [[] for _ in range(batch)]
        self.len = [0] * batch
        self.refs = np.zeros(pages, dtype=np.int64)

    def table(self):
        t = np.full((self.batch, self.max_pages), -1, dtype=np.int32)
        for b, r in enumerate(self.rows):
            t[b, : len(r)] = r
        return t

    def _free(self):
        return list(np.flatnonzero(self.refs == 0))

    def reserve(self, n_new):
        ok, free, cut = [0] * self.batch, self._free(), False
        for b in range(self.batch):
            hold = -(-(self.len[b] + n_new[b]) // self.page)
            if n_new[b] < 0 or hold > self.max_pages:
                continue
            need = max(0, hold - len(self.rows[b]))
            if need and (cut or need > len(free)):
                cut = True
                continue
            for _ in range(need):
                p = free.pop(0)
                self.refs[p] = 1
                self.rows[b].append(int(p))
            ok[b] = 1
        return ok

    def alone(self, b, lo, hi):
        """Does the row hold, alone, the pages of positions lo .. hi - 1?"""
        js = range(lo // self.page, -(-hi // self.page))
        return all(j < len(self.rows[b]) and self.refs[self.rows[b][j]] == 1 for j in js)

    def append(self, layer, k, v, n_new):
        """k, v float64 [batch, T, heads, dim]; returns whether a value was out of range."""
        odd = False
        for b in range(self.batch):
            n, L = n_new[b], self.len[b]
            if n <= 0 or not self.alone(b, L, L + n):
                continue
            for kv, x in ((0, k), (1, v)):
                for j in range(L // self.page, -(-(L + n) // self.page)):
                    p = self.rows[b][j]
                    lo, hi = max(L, j * self.page), min(L + n, (j + 1) * self.page)
                    off = lo - j * self.page
                    for h in range(self.heads):
                        y = x[b, lo - L: hi - L, h]
                        good = np.abs(y) <= XMAX
                        odd = odd or not good.all()
                        s = scale_for(np.abs(np.where(good, y, 0.0)).max())
                        blk = self.q[kv, layer, p, h]
                        if off:
                            old = self.s[kv, layer, p, h]
                            s = max(s, old)
                            blk[:off] = e4m3(blk[:off] * (old / s))
                        with np.errstate(invalid="ignore"):
                            blk[off: off + hi - lo] = e4m3(y / s)
                        self.s[kv, layer, p, h] = s
        return odd

    def values(self, kv, layer, b, lo, hi):
        """Positions lo .. hi - 1 of a row: [hi - lo, heads, dim]."""
        out = np.zeros((hi - lo, self.heads, self.dim))
        for t in range(lo, hi):
            p = self.rows[b][t // self.page]
            out[t - lo] = self.q[kv, layer, p, :, t % self.page] \
                * self.s[kv, layer, p][:, None]
        return out

    def commit(self, accepted, path=None):
        for b in range(self.batch):
            L, n = self.len[b], accepted[b] + 1
            idx = [0] + (list(path[b][: n - 1]) if path is not None else list(range(1, n)))
            idx = [int(i) for i in idx[:n]]
            if any(i != m for m, i in enumerate(idx)):
                at = [(self.rows[b][(L + i) // self.page], (L + i) % self.page) for i in idx]
                to = [(self.rows[b][(L + m) // self.page], (L + m) % self.page)
                      for m in range(n)]
                for kv in range(2):
                    for ly in range(self.layers):
                        q, s = self.q[kv, ly], self.s[kv, ly]
                        val = [q[p, :, i].copy() for p, i in at]
                        src = [s[p].copy() for p, _ in at]
                        for p in dict.fromkeys(p for p, _ in to):
                            mine = [m for m in range(n) if to[m][0] == p]
                            new = np.max([src[m] for m in mine], axis=0)
                            off = L % self.page if p == to[0][0] else 0
                            if off:
                                new = np.maximum(new, s[p])
                                q[p, :, :off] = e4m3(q[p, :, :off]
                                                     * (s[p] / new)[:, None, None])
                            for m in mine:
                                q[p, :, to[m][1]] = e4m3(val[m] * (src[m] / new)[:, None])
                            s[p] = new
            self.len[b] = L + n
            while len(self.rows[b]) > -(-self.len[b] // self.page):
                self.refs[self.rows[b].pop()] -= 1

    def fork(self, src):
        old, length, ok = [list(r) for r in self.rows], list(self.len), [1] * self.batch
        takers = [[b for b in range(self.batch) if src[b] == i] for i in range(self.batch)]
        keeper = [None if not t else (i if i in t else t[0]) for i, t in enumerate(takers)]
        for i in range(self.batch):
            full = length[i] // self.page
            for j, p in enumerate(old[i]):
                self.refs[p] += len(takers[i]) - 1 if j < full else (0 if takers[i] else -1)
        free = self._free()
        for b in range(self.batch):
            s = src[b]
            if s < 0:
                self.rows[b], self.len[b] = [], 0
            elif keeper[s] == b:
                self.rows[b], self.len[b] = list(old[s]), length[s]
            else:
                full, tail = length[s] // self.page, length[s] % self.page
                self.rows[b], self.len[b] = old[s][:full], length[s]
                if not tail:
                    continue
                if not free:
                    ok[b], self.len[b] = 0, full * self.page
                    continue
                p, f = int(free.pop(0)), old[s][full]
                self.refs[p] = 1
                self.q[:, :, p, :, :tail] = self.q[:, :, f, :, :tail]
                self.s[:, :, p] = self.s[:, :, f]
                self.rows[b].append(p)
        return ok


def visible(L, n, t, parent=None, window=0, sinks=0):
    """Positions that query t of a block of n sees, as a mask over L + n."""
    chain = [t]
    while chain[-1] > 0:
        chain.append(chain[-1] - 1 if parent is None else int(parent[chain[-1]]))
    pos = L + len(chain) - 1
    see = np.zeros(L + n, dtype=bool)
    j = np.arange(L)
    see[:L] = True if not window else (pos - j < window) | (j < sinks)
    for up, i in enumerate(chain):
        see[L + i] = not window or up < window or L + i < sinks
    return see


def attend(q, k, v, L, n, scale, parent=None, window=0, sinks=0):
    """One row: q [T, q_heads, dim], k, v [L + n, heads, dim] float64. Returns out, lse, the
    weighted mean of |v| and the largest sums |q| |k| and max|q| sum|k| behind a score."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    o, av = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -math.inf)
    ab, qk = np.zeros((T, Hq)), np.zeros((T, Hq))
    for t in range(n):
        see = visible(L, n, t, parent, window, sinks)
        for h in range(H):
            kk, vv, qq = k[see, h], v[see, h], q[t, h * G:(h + 1) * G]
            if not len(kk):
                continue
            s = qq @ kk.T * scale
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            den = e.sum(-1, keepdims=True)
            w = e / den
            sl = slice(h * G, (h + 1) * G)
            o[t, sl], av[t, sl] = w @ vv, w @ np.abs(vv)
            lse[t, sl] = (np.log(den) + m)[:, 0]
            ab[t, sl] = (np.abs(qq) @ np.abs(kk).T).max(-1)
            qk[t, sl] = np.abs(qq).max(-1) * np.abs(kk).sum(-1).max()
    return o, lse, av, ab, qk
