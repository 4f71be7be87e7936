"""The paged 4-bit cache in plain numpy and 64 bits: what the CUDA operators are tested
against.  Tables are lists, a page's tokens are bytes placed one by one by formula; no
code is shared with the library."""
import math

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([MAGNITUDES, -MAGNITUDES])
# e4m3 without its NaN (127): exponent 4 bits, mantissa 3, subnormals below 2^-6
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def _nearest(x, grid):
    """Index of the nearest grid value (grid ascending, x >= 0), ties to the even index, saturating."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)


def quantise(x, exp):
    """x [..., d] -> codes [..., d] (uint8), scale bytes [..., d / 16], held values [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    top = np.abs(b).max(-1)
    s = _nearest(np.minimum(top / 6 / 2.0 ** exp, 448.0), E4M3)
    S = (E4M3[s] * 2.0 ** exp)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(S > 0, np.abs(b) / S, 0.0)
    code = _nearest(t, MAGNITUDES) + 8 * np.signbit(b)
    held = E2M1[code] * S
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8), held.reshape(x.shape)


def page_bytes(P, d):
    return P * d * 9 // 8


def put_token(page, P, d, t, kc, ks, vc, vs):
    """Token t's codes and scales into a page's bytes (uint8 [P d 9/8])."""
    b = min(P, 64)
    blk = page[(t // b) * (b * d * 9 // 8):]
    u = t % b
    for c in range(d):
        _half(blk, u * (d // 2) + c // 2, c % 2, kc[c])
        at = b * d * 9 // 16 + (((u // 8) * (d // 16) + c // 16) * 4 + u % 8 // 2) * 16 + c % 16
        _half(blk, at, u % 2, vc[c])
    for g in range(d // 16):
        blk[b * d // 2 + u * (d // 16) + g] = ks[g]
        blk[b * d * 17 // 16 + (((u // 8) * (d // 16) + g) * 4 + u % 8 // 2) * 2 + u % 2] = vs[g]


def _half(a, at, high, code):
    a[at] = (a[at] & 0x0F) | (code << 4) if high else (a[at] & 0xF0) | code


def summary(keys):
    """Held keys [n, d] of a page (units of 2^k_exp) -> (largest int8 [d], smallest int8 [d], e)."""
    hi, lo = keys.max(0), keys.min(0)
    m = max(np.abs(hi).max(), np.abs(lo).max())
    e = math.frexp(m)[1] - 7 if m > 0 else 0
    return np.ceil(hi * 2.0 ** -e).astype(np.int8), np.floor(lo * 2.0 ** -e).astype(np.int8), e


class Model:
    """Rows, pages and counts, and every row's held keys and values (one layer)."""

    def __init__(self, n_pages, P, R, M):
        self.n, self.P, self.R, self.M = n_pages, P, R, M
        self.table = [[] for _ in range(R)]
        self.length = [0] * R
        self.refs = [0] * n_pages
        self.copies = []

    def pages(self, n):
        return -(-n // self.P)

    def resize(self, rows, lens):
        """False (and nothing changed) where the pool is too small or an argument is wrong."""
        todo = [(r, n) for r, n in zip(rows, lens) if r >= 0]
        if len({r for r, _ in todo}) < len(todo) or any(r >= self.R or not 0 <= n <= self.M * self.P for r, n in todo):
            return False
        refs, table = list(self.refs), [list(t) for t in self.table]
        for r, n in todo:
            while len(table[r]) > self.pages(n):
                refs[table[r].pop()] -= 1
        at = {r: table[r][-1] for r, n in todo if n > self.length[r] and self.length[r] % self.P}
        free = [i for i in range(self.n) if refs[i] == 0]
        copies, want = [], 0
        hold = list(refs)
        for r, n in todo:
            p = at.get(r)
            if p is not None and hold[p] > 1:
                hold[p] -= 1
                copies.append((r, p))
                want += 1
            want += max(0, self.pages(n) - len(table[r]))
        if want > len(free):
            return False
        self.copies = []
        for r, n in todo:
            if (r, at.get(r)) in copies:
                q = free.pop(0)
                refs[at[r]] -= 1
                refs[q] = 1
                self.copies.append((at[r], q))
                table[r][-1] = q
            while len(table[r]) < self.pages(n):
                q = free.pop(0)
                refs[q] = 1
                table[r].append(q)
        self.refs, self.table = refs, table
        for r, n in todo:
            self.length[r] = n
        return True

    def fork(self, src, dst):
        todo = [(s, d) for s, d in zip(src, dst) if s >= 0 and d >= 0]
        to = [d for _, d in todo]
        if any(x >= self.R for p in todo for x in p) or len(set(to)) < len(to) or any(s in to for s, _ in todo) or any(
                self.length[d] for d in to):
            return False
        for s, d in todo:
            self.table[d], self.length[d] = list(self.table[s]), self.length[s]
            for p in self.table[s]:
                self.refs[p] += 1
        return True

    def compact(self):
        live = [i for i in range(self.n) if self.refs[i] > 0]
        n = len(live)
        src, dst = [i for i in live if i >= n], [i for i in range(n) if self.refs[i] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(p, p) for p in t] for t in self.table]
        self.copies = list(to.items())
        return True


def attend(q, k, v, visible, scale):
    """out [n, d], lse [n] of queries q [n, d] over k, v [m, d] where visible [n, m]."""
    out, lse = np.zeros((q.shape[0], v.shape[-1])), np.full(q.shape[0], -np.inf)
    z = q @ k.T * scale
    for i in range(q.shape[0]):
        if visible[i].any():
            zi = z[i][visible[i]]
            w = np.exp(zi - zi.max())
            out[i] = w @ v[visible[i]] / w.sum()
            lse[i] = zi.max() + math.log(w.sum())
    return out, lse


def choose(q, sums, n, keep, first, last):
    """q [G, d] (64 bits), sums: (largest, smallest, e) of the row's pages -> chosen ordinals, ascending."""
    if n <= keep:
        return list(range(n))
    hi, lo = np.float32(np.maximum(q, 0).sum(0)), np.float32(np.minimum(q, 0).sum(0))
    top = np.float32(max(hi.max(), (-lo).max()))
    inv = np.float32(127) / top if top > 0 else np.float32(0)
    hi, lo = np.rint(hi * inv).astype(np.int64), np.rint(lo * inv).astype(np.int64)
    score = [math.inf if j < first or j >= n - last else float(hi @ sums[j][0].astype(np.int64) + lo @ sums[j][1].astype(np.int64)) * 2.0 ** sums[j][2]
             for j in range(n)]
    return sorted(sorted(range(n), key=lambda j: (-score[j], j))[:keep])
