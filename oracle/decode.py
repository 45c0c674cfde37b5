"""Float64 definitions of the decode operators: cache pages, attention of one token, logits.

Written from the definitions alone (plain loops, one sequence after the other); it shares no
code with the CUDA path. Pages are handed out one at a time from the lowest free number.
"""

from __future__ import annotations

import numpy as np


class Pool:
    """A cache's bookkeeping and contents: table, lens, refs as lists, k and v as
    [layers, pages, kv_heads, page, dim] arrays."""

    def __init__(self, table, lens, refs, k, v):
        self.table = [list(map(int, r)) for r in table]
        self.lens = list(map(int, lens))
        self.refs = list(map(int, refs))
        self.k, self.v = np.array(k), np.array(v)
        self.page = self.k.shape[3]
        self.cols = len(self.table[0])
        self.bad = self.no_page = False

    def held(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, seq, add):
        free, asked, seen = self.free_pages(), 0, set()
        for s, n in zip(seq, add):
            if not 0 <= s < len(self.lens) or s in seen or n < 0:
                self.bad = True
                continue
            seen.add(s)
            old, new = self.lens[s], self.lens[s] + n
            if new > self.cols * self.page:
                self.no_page = True
                continue
            need = self.held(new) - self.held(old)
            first = asked
            asked += need
            if need and asked > len(free):
                self.no_page = True
                continue
            for i in range(need):
                self.table[s][self.held(old) + i] = free[first + i]
                self.refs[free[first + i]] = 1
            self.lens[s] = new

    def release(self, s):
        for j in range(self.held(self.lens[s])):
            self.refs[self.table[s][j]] -= 1
            self.table[s][j] = -1
        self.lens[s] = 0

    def free(self, seq):
        for s in seq:
            if not 0 <= s < len(self.lens):
                self.bad = True
                continue
            self.release(s)

    def fork(self, src, dst):
        n = len(self.lens)
        named = {d for d in dst if 0 <= d < n}
        pairs, seen = [], set()
        for s, d in zip(src, dst):
            ok = 0 <= s < n and 0 <= d < n and s not in named and d not in seen
            if 0 <= d < n:
                seen.add(d)
            if ok:
                pairs.append((s, d))
            else:
                self.bad = True
        for s, d in pairs:
            self.release(d)
            for j in range(self.lens[s] // self.page):
                self.refs[self.table[s][j]] += 1
        free = self.free_pages()
        for s, d in pairs:
            full, part = divmod(self.lens[s], self.page)
            self.table[d] = self.table[s][:full] + [-1] * (self.cols - full)
            self.lens[d] = self.lens[s]
            if not part:
                continue
            if not free:
                self.no_page = True
                for j in range(full):
                    self.refs[self.table[d][j]] -= 1
                self.table[d] = [-1] * self.cols
                self.lens[d] = 0
                continue
            p = free.pop(0)
            self.table[d][full] = p
            self.refs[p] = 1
            for x in (self.k, self.v):
                x[:, p, :, :part] = x[:, self.table[s][full], :, :part]

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(len(self.refs) - 1, live - 1, -1) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
        for s, row in enumerate(self.table):
            for j in range(self.held(self.lens[s])):
                row[j] = to.get(row[j], row[j])
        return live

    def position(self, s, t):
        return self.table[s][t // self.page], t % self.page

    def write(self, layer, k, v, seq, start):
        for i, s in enumerate(seq):
            for t in range(start[i], start[i + 1]):
                pos = self.lens[s] - (start[i + 1] - t) if 0 <= s < len(self.lens) else -1
                if pos < 0:
                    self.bad = True
                    continue
                p, r = self.position(s, pos)
                self.k[layer, p, :, r], self.v[layer, p, :, r] = k[t], v[t]


def visible(n, window, sinks):
    """The positions a new token at the end of n tokens attends to."""
    if window == 0:
        return list(range(n))
    return [j for j in range(n) if j < sinks or j >= n - window]


def attention(q, k, v, scale):
    """q [H, D], k and v [n, Hkv, D] (visible positions): out [H, D], lse [H], and per element
    of out the weighted sum of |v| and per head the largest sum of |q k| (for error bounds)."""
    H, D = q.shape
    n, Hkv = k.shape[:2]
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    mass, reach = np.zeros((H, D)), np.zeros(H)
    if n == 0:
        return out, lse, mass, reach
    for h in range(H):
        g = h // (H // Hkv)
        s = scale * (k[:, g] @ q[h])
        top = s.max()
        w = np.exp(s - top)
        out[h] = w @ v[:, g] / w.sum()
        lse[h] = top + np.log(w.sum())
        mass[h] = w @ np.abs(v[:, g]) / w.sum()
        reach[h] = abs(scale) * (np.abs(k[:, g]) @ np.abs(q[h])).max()
    return out, lse, mass, reach


def guided_logits(cond, uncond=None, scale=1.0, bias=None, tokens=(), prompt=0, repetition=1.0,
                  frequency=0.0, presence=0.0, temperature=1.0, allowed=None, noise=None):
    """One row: (z, token, logprob, size), size the magnitude that each z's roundings scale with."""
    V = len(cond)
    z = np.array(cond, dtype=np.float64)
    size = np.where(np.isfinite(z), np.abs(z), 0.0)
    if uncond is not None and scale != 1.0:
        u = np.array(uncond, dtype=np.float64)
        both = np.isfinite(z) & np.isfinite(u)
        z[both] = u[both] + scale * (z[both] - u[both])
        size[both] = abs(scale) * np.abs(np.array(cond)[both]) + abs(1 - scale) * np.abs(u[both])
    if bias is not None:
        z = z + bias
        size = size + np.abs(bias)
    count, seen = np.zeros(V), np.zeros(V, bool)
    for t, x in enumerate(tokens):
        if 0 <= x < V:
            seen[x] = True
            count[x] += t >= prompt
    with np.errstate(invalid="ignore"):
        z = np.where(seen, np.where(z > 0, z / repetition, z * repetition), z)
    size = size * np.where(seen, max(repetition, 1.0), 1.0)
    z = z - (frequency * count + presence * (count > 0))
    size = size + abs(frequency) * count + abs(presence)
    if temperature > 0:
        z, size = z / temperature, size / temperature
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
    pick = z + noise if noise is not None and temperature > 0 else z
    pick = np.where(z > -np.inf, pick, -np.inf)
    if not (pick > -np.inf).any():
        return z, -1, -np.inf, size, pick
    token = int(np.flatnonzero(pick == np.nanmax(pick))[0])
    top = np.nanmax(z)
    return z, token, z[token] - top - np.log(np.exp(z - top).sum()), size, pick
