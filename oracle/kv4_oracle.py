"""fp64 restatement of the paged 4-bit context cache: values, attention, page operations.

Written from the definitions: e2m1 and e4m3 as tables of numbers, rounding as
a nearest-number search with ties to the even code, pages as Python lists.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite non-negative e4m3 number, in the order of its code 0x00..0x7E
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8) if not (e == 15 and m == 7)])


def nearest_code(y, table):
    """Code of the table number nearest to each y >= 0 (beyond the last: the last); ties to the even code."""
    y = np.asarray(y, np.float64)
    hi = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
    lo = hi - 1
    d_lo, d_hi = y - table[lo], table[hi] - y
    even = np.where(lo % 2 == 0, lo, hi)
    return np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, even))


def kv4_values(x, e):
    """What rows x [..., hd] read back as from the cache with exponent e."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    bad = ~np.isfinite(g).all(-1, keepdims=True)
    g = np.where(np.isfinite(g), g, 0.0) * 2.0 ** -e
    s = np.maximum(E4M3[nearest_code(np.minimum(np.abs(g).max(-1, keepdims=True) / 6.0, 448.0), E4M3)], 2.0 ** -9)
    v = np.sign(g) * E2M1[nearest_code(np.abs(g) / s, E2M1)] * s * 2.0 ** e
    return np.where(bad, np.nan, v).reshape(x.shape)


def paged_attn(q, kc, vc, kb, vb):
    """One sequence: q [B][Hq][hd], cached kc, vc [T][Hkv][hd], block kb, vb [B][Hkv][hd].

    Returns O [B][Hq][hd] and, for error bounds, sum p |v| / sum p over the
    cached and over the block's keys, and the largest |score|.
    """
    q, kc, vc, kb, vb = (np.asarray(a, np.float64) for a in (q, kc, vc, kb, vb))
    B, Hq, hd = q.shape
    T, Hkv = kc.shape[:2]
    G = Hq // Hkv
    O, Ac, Ab = np.empty((B, Hq, hd)), np.empty((B, Hq, hd)), np.empty((B, Hq, hd))
    smax = 0.0
    for h in range(Hq):
        k = np.concatenate([kc[:, h // G], kb[:, h // G]])
        v = np.concatenate([vc[:, h // G], vb[:, h // G]])
        s = q[:, h] @ k.T / np.sqrt(hd)
        smax = max(smax, float(np.abs(s).max())) if np.isfinite(s).all() else smax
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        O[:, h] = p @ v
        Ac[:, h], Ab[:, h] = p[:, :T] @ np.abs(v[:T]), p[:, T:] @ np.abs(v[T:])
    return O, Ac, Ab, smax


class PageBook:
    """Tables, lengths and counts of N sequences over a pool, one list operation at a time."""

    def __init__(self, table, length, ref, page):
        self.table, self.len, self.ref = np.array(table), np.array(length), np.array(ref)
        self.page = page

    def pages(self, n, length=None):
        return -(-int(self.len[n] if length is None else length) // self.page)

    def reserve(self, n_new):
        """Returns (start, copies) with copies a list of (source, destination) pages."""
        free = [p for p in range(len(self.ref)) if self.ref[p] <= 0]
        before = self.ref.copy()
        start, copies, asked = np.full(len(self.len), -1, np.int32), [], 0
        for n, m in enumerate(n_new):
            m, have = int(m), self.pages(n)
            want = self.pages(n, int(self.len[n]) + m)
            cow = m > 0 and self.len[n] % self.page != 0 and before[self.table[n][have - 1]] > 1
            need = want - have + int(cow)
            asked += need
            if need > 0 and asked > len(free):
                continue
            got = free[asked - need:asked]
            if cow:
                old = self.table[n][have - 1]
                copies.append((int(old), got[0]))
                self.ref[old] -= 1
                self.table[n][have - 1] = got[0]
            self.table[n][have:want] = got[int(cow):]
            self.ref[got] = 1
            start[n] = self.len[n]
            self.len[n] += m
        return start, copies

    def remap(self, parent, keep=None):
        table, length = self.table.copy(), self.len.copy()
        for n, p in enumerate(parent):
            row = np.full(table.shape[1], -1)
            l = 0
            if p >= 0:
                l = int(length[p]) if keep is None or keep[n] < 0 else min(int(length[p]), int(keep[n]))
                row[:self.pages(n, l)] = table[p][:self.pages(n, l)]
            for x in table[n]:
                if x >= 0:
                    self.ref[x] -= 1
            for x in row:
                if x >= 0:
                    self.ref[x] += 1
            self.table[n], self.len[n] = row, l

    def compact(self):
        """Returns (map, live, moves)."""
        used = [p for p in range(len(self.ref)) if self.ref[p] > 0]
        live = len(used)
        holes = [p for p in range(live) if self.ref[p] <= 0]
        moves = list(zip([p for p in used if p >= live], holes))
        m = np.full(len(self.ref), -1, np.int32)
        m[used] = used
        for s, d in moves:
            m[s], self.ref[d], self.ref[s] = d, self.ref[s], 0
        self.table = np.where(self.table >= 0, m[self.table], self.table)
        return m, live, moves
