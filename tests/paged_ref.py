"""Plain 64-bit forms of the paged-cache operators, in numpy, and a list-based model of the pages' books.

Written from the definitions in include/lsa.h; shares no code with the library.
"""
import numpy as np
import torch


def values(x, scale=None):
    """A cache tensor [n_pages, page_size, Hkv, D] in 64 bits."""
    y = x.detach().cpu().float().numpy().astype(np.float64)
    return y if scale is None else y * scale.cpu().numpy().astype(np.float64)[..., None]


def attention(q, k, v, table, lens, page_size, window, scale):
    """out [B, Hq, D], lse [B, Hq], and per (b, j) the largest sum of |q k| and the number of entries, for bounds."""
    B, Hq, D = q.shape
    n_pages, _, Hkv, _ = k.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mag, vmax = np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        n = int(min(max(lens[b], 0), table.shape[1] * page_size))
        t = np.arange(max(0, n - window) if window else 0, n)
        page = table[b, t // page_size].astype(np.int64)
        ok = (page >= 0) & (page < n_pages)
        t, page = t[ok], page[ok]
        if not len(t):
            continue
        K, V = k[page, t % page_size], v[page, t % page_size]
        for j in range(Hq):
            h = j // G
            with np.errstate(invalid="ignore", over="ignore"):
                a = scale * (K[:, h] @ q[b, j])
                mag[b, j] = scale * np.max(np.abs(K[:, h]) @ np.abs(q[b, j]))
                vmax[b, j] = np.max(np.abs(V[:, h]))
                m = a.max()
                if m == -np.inf:
                    continue
                w = np.exp(a - m)
                out[b, j] = (w @ V[:, h]) / w.sum()
                lse[b, j] = m + np.log(w.sum())
    return out, lse, mag, vmax


def norm_rope(x, w, eps, pos, freq, rot, interleaved, inverse, mscale):
    """x [T, H, D] -> y, and the bound of |a| + |b| of each element's pair."""
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    size = np.abs(y)
    if rot:
        phi = pos.astype(np.float64)[:, None, None] * freq * (-1.0 if inverse else 1.0)
        c, s = mscale * np.cos(phi), mscale * np.sin(phi)
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia] = size[..., ib] = mscale * (np.abs(a) + np.abs(b))
    return y, size


class Books:
    """The pages' books as lists, every rule spelled out."""

    def __init__(self, n_rows, max_pages, n_pages, page_size):
        self.rows, self.max_pages, self.n_pages, self.ps = [[] for _ in range(n_rows)], max_pages, n_pages, page_size
        self.len, self.refs = [0] * n_rows, [0] * n_pages

    def pages(self, n):
        return -(-n // self.ps)

    def _free(self):
        return [p for p in range(self.n_pages) if self.refs[p] == 0]

    def grow(self, add):
        need = [self.pages(n + max(0, a)) - self.pages(n) for n, a in zip(self.len, add)]
        free = self._free()
        if any(n + max(0, a) > self.max_pages * self.ps for n, a in zip(self.len, add)) or sum(need) > len(free):
            return "capacity"
        for r, a in enumerate(add):
            for _ in range(need[r]):
                p = free.pop(0)
                self.refs[p] = 1
                self.rows[r].append(p)
            self.len[r] += max(0, a)
        return None

    def fork(self, src, dst):
        none = [-1] * len(src)
        n = len(self.rows)
        if any(not 0 <= r < n for r in src + dst) or any(self.len[d] for d in dst) or len(set(dst)) < len(dst) \
                or set(src) & set(dst):
            return "invalid", none, none
        free = self._free()
        if sum(self.len[s] % self.ps > 0 for s in src) > len(free):
            return "capacity", none, none
        cs, cd = [], []
        for s, d in zip(src, dst):
            full = self.len[s] // self.ps
            row = self.rows[s][:full]
            for p in row:
                self.refs[p] += 1
            cs.append(-1)
            cd.append(-1)
            if self.len[s] % self.ps:
                cs[-1], cd[-1] = self.rows[s][full], free.pop(0)
                self.refs[cd[-1]] = 1
                row = row + [cd[-1]]
            self.rows[d], self.len[d] = list(row), self.len[s]
        return None, cs, cd

    def free(self, rows):
        bad = False
        for r in rows:
            if not 0 <= r < len(self.rows):
                bad = True
                continue
            for p in self.rows[r]:
                self.refs[p] -= 1
            self.rows[r], self.len[r] = [], 0
        return "invalid" if bad else None

    def compact(self):
        held = sum(r > 0 for r in self.refs)
        src = [p for p in range(held, self.n_pages) if self.refs[p] > 0]
        dst = [p for p in range(held) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.rows = [[to.get(p, p) for p in row] for row in self.rows]
        pad = [-1] * (self.n_pages - len(src))
        return src + pad, dst + pad, len(src)

    def table(self):
        return np.array([r + [-1] * (self.max_pages - len(r)) for r in self.rows], np.int32)


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x, np.int32), device=device)
