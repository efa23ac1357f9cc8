"""Oracle: the paged FP8 KV cache (test infrastructure), plain NumPy and Python in 64 bits.

Pages "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson AGX
Thor", sections "Using NVFP4 quantization to accelerate Qwen3.6-27B inference" (the KV cache is
FP8), "Using tree-based multi-token prediction to accelerate LLM inference" (one pass over the
drafted tree) and "Reusing KV cache across agent turns" (turns share cached pages).

* Token t of sequence b is slot t % page of page table[b][t // page]; a page is [H][page][D] E4M3
  bytes.  A token outside the table, or on a page id outside the cache, does not exist.
* append: node v of sequence b is encoded (oracle/kvfp8.py) at token lens[b] + v, v < counts[b].
* attention: node v sees the tokens before lens[b], and of the nodes itself and its ancestors (with
  parents; a parent outside [0, v) makes v a root) or the nodes 0 .. v (without); softmax of
  sm_scale * q . k_hat over what it sees, times v_hat.  A row that sees nothing gives zeros and
  -infinity.
* compact: token lens[b] + path[i] moves to lens[b] + 1 + i; the new length is lens[b] + 1 + L.
* resize, fork: the pool as include/nvfp4.h states it, entry by entry.

Parity unpinned by the pages: they name neither page layout nor attention shapes.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import kvfp8 as KV


def _slot(pages, table, b, t):
    """(page id, slot) of token t of sequence b, or None where it does not exist."""
    P, _, page, _ = pages.shape[-4:]
    if t < 0 or t // page >= table.shape[1]:
        return None
    p = int(table[b, t // page])
    return (p, t % page) if 0 <= p < P else None


def _count(counts, b, M):
    return M if counts is None else max(0, min(M, int(counts[b])))


def append(x, scale, pages, table, lens, counts=None):
    """pages [P, H, page, D] with x [B, M, H, D] (float32 values) written into it: a new array."""
    out = pages.copy()
    B, M = x.shape[:2]
    for b in range(B):
        if lens[b] < 0:
            continue
        for v in range(_count(counts, b, M)):
            at = _slot(pages, table, b, int(lens[b]) + v)
            if at is not None:
                out[at[0], :, at[1]] = KV.encode(x[b, v], scale)
    return out


def ancestors(parent):
    """[M, M] bool: node u is v or an ancestor of v."""
    M = len(parent)
    line = np.zeros((M, M), dtype=bool)
    for v in range(M):
        u = v
        while True:
            line[v, u] = True
            p = int(parent[u])
            if not 0 <= p < u:
                break
            u = p
    return line


def attention(q, k_pages, v_pages, k_scale, v_scale, table, lens, parent=None, counts=None, sm_scale=None):
    """q [B, M, Hq, D] -> (out float64 [B, M, Hq, D], lse float64 [B, M, Hq],
    size float64 [B, M, Hq, D]: the softmax's mean of |v_hat|, the scale of the sums' rounding)."""
    B, M, Hq, D = q.shape
    H = k_pages.shape[1]
    G = Hq // H
    sm = 1.0 / np.sqrt(D) if sm_scale is None else float(np.float32(sm_scale))
    out, size = np.zeros((B, M, Hq, D)), np.zeros((B, M, Hq, D))
    lse = np.full((B, M, Hq), -np.inf)
    for b in range(B):
        if lens[b] < 0:
            continue
        n, c = int(lens[b]), _count(counts, b, M)
        slots = [_slot(k_pages, table, b, t) for t in range(n + c)]
        there = np.array([s is not None for s in slots], dtype=bool)
        at = np.array([s or (0, 0) for s in slots], dtype=np.int64).reshape(-1, 2)
        seen = np.zeros((M, n + c), dtype=bool)
        line = np.tri(M, dtype=bool) if parent is None else ancestors(parent[b])
        for v in range(c):
            seen[v, :n] = True
            seen[v, n:] = line[v, :c]
        seen &= there
        for h in range(H):
            k = F.decode_e4m3(k_pages[at[:, 0], h, at[:, 1]]) * float(k_scale)
            x = F.decode_e4m3(v_pages[at[:, 0], h, at[:, 1]]) * float(v_scale)
            for j in range(h * G, (h + 1) * G):
                for v in range(c):
                    w = seen[v]
                    if not w.any():
                        continue
                    z = sm * (k[w] @ q[b, v, j].astype(np.float64))
                    top = z.max()
                    e = np.exp(z - top)
                    lse[b, v, j] = top + np.log(e.sum())
                    out[b, v, j] = e @ x[w] / e.sum()
                    size[b, v, j] = e @ np.abs(x[w]) / e.sum()
    return out, lse, size


def compact(pages, table, lens, result):
    """pages [L, P, H, page, D] with the accepted paths moved (a new array), and the new lengths."""
    out = pages.copy()
    M = result.shape[1] - 3
    new = lens.copy()
    for b in range(len(lens)):
        if lens[b] < 0:
            continue
        n = max(0, min(M - 1, int(result[b, 1])))
        new[b] = lens[b] + 1 + n
        for i in range(n):
            v = int(result[b, 3 + i])
            if not 0 <= v < M:
                continue
            x, y = _slot(pages, table, b, int(lens[b]) + v), _slot(pages, table, b, int(lens[b]) + 1 + i)
            if x is not None and y is not None:
                out[:, y[0], :, y[1]] = pages[:, x[0], :, x[1]]
    return out, new


class Pool:
    """The page pool, entry by entry (include/nvfp4.h)."""

    def __init__(self, seqs, width, pages):
        self.table = np.full((seqs, width), -1, dtype=np.int32)
        self.held = np.zeros(seqs, dtype=np.int32)
        self.refs = np.zeros(pages, dtype=np.int32)
        self.free = list(range(pages - 1, -1, -1))

    def writable(self, seq, page, lo, hi):
        """Whether tokens lo .. hi - 1 of a sequence lie on pages that no other sequence holds."""
        return all(self.refs[p] == 1 for p in self.table[seq, lo // page: -(-hi // page)] if p >= 0)

    def _give_up(self, pages):
        for p in pages:
            self.refs[p] -= 1
        done = set()
        for p in pages:
            if self.refs[p] == 0 and p not in done:
                done.add(p)
                self.free.append(p)

    def resize(self, page, seqs, tokens):
        S, W = self.table.shape
        plan, named = [], set()
        for s, t in zip(map(int, seqs), map(int, tokens)):
            need = -(-t // page)
            if 0 <= s < S and t >= 0 and need <= W and s not in named:
                plan.append((s, need))
            named.add(s)
        want = sum(max(0, need - self.held[s]) for s, need in plan)
        if want > len(self.free):
            return int(want - len(self.free))
        dropped = []
        for s, need in plan:
            for i in range(self.held[s], need):
                p = self.free.pop()
                self.table[s, i] = p
                self.refs[p] = 1
            for i in range(need, self.held[s]):
                dropped.append(int(self.table[s, i]))
                self.table[s, i] = -1
            self.held[s] = need
        self._give_up(dropped)
        return 0

    def fork(self, page, src, dst, tokens):
        """Returns (shortage, [(page to copy, to, used slots)])."""
        S = self.table.shape[0]
        plan, named = [], set()
        every = set(map(int, dst))
        for s, d, t in zip(map(int, src), map(int, dst), map(int, tokens)):
            if 0 <= s < S and 0 <= d < S and t >= 0 and d not in named and s not in every and \
                    -(-t // page) <= self.held[s]:
                plan.append((s, d, t))
            named.add(d)
        want = sum(t % page > 0 for _, _, t in plan)
        if want > len(self.free):
            return want - len(self.free), []
        moves, dropped, rows = [], [], []
        for s, d, t in plan:
            row = [int(p) for p in self.table[s, : t // page]]
            for p in row:
                self.refs[p] += 1
            if t % page:
                p = self.free.pop()
                self.refs[p] = 1
                moves.append((int(self.table[s, t // page]), p, t % page))
                row.append(p)
            rows.append(row)
            dropped += [int(p) for p in self.table[d, : self.held[d]]]
        self._give_up(dropped)
        for (s, d, t), row in zip(plan, rows):
            self.table[d] = -1
            self.table[d, : len(row)] = row
            self.held[d] = len(row)
        return 0, moves


def copy_slots(pages, moves):
    """pages [L, P, H, page, D] after a fork's moves: a new array."""
    out = pages.copy()
    for x, y, n in moves:
        out[:, y, :, :n] = pages[:, x, :, :n]
    return out
