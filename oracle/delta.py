"""Oracle: the gated delta rule (test infrastructure), plain NumPy in 64 bits, token by token.

Page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson AGX Thor", section "Reusing
KV cache across agent turns": the model is a hybrid, whose recurrent states are kept and restored with its cached pages.

Per value head, S [Dv, Dk]: S <- e^g S, u = beta (v - S k), S <- S + u k^T, o = scale S q; value head h uses key head
h // (H // Hk); q and k are divided by sqrt(sum of squares + eps) where eps is not None.

* chain: sequence b begins with slot src[b] (-1: zeros; below -1 or past the slots: not in use) and leaves its state in
  slot dst[b], unless that is out of range, the src of another sequence in use, or the dst of an earlier one.
* tree: a node goes on from its parent's state (outside [0, v): from the sequence's).
* commit: a state taken through node 0 and the path's nodes with the u and k of the tree.

`Bounds` follows the rounding of an implementation.  With u = 2^-22 (the bits that factors of a state keep), a row of S
is off by at most e in 2-norm: a token multiplies e by e^g max(1, |1 - beta |k|^2|), the norm of what it does to a row,
and adds the rounding of its sums, (Dk + 80) u times the size of what is summed.  `big` is the recurrence of absolute
values, e^g big + |u| |k|^T: however the sum that is S was split into blocks, big is no less than the sum of the parts'
sizes.

Parity unpinned by the pages: they name no recurrence.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -22


def normalised(x, eps):
    x = x.astype(np.float64)
    return x if eps is None else x / np.sqrt((x ** 2).sum(-1, keepdims=True) + eps)


class Bounds:
    """A state [H, Dv, Dk] on its way, with how far an implementation may be off (e [H, Dv]) and big."""

    def __init__(self, state):
        self.s = state.astype(np.float64).copy()
        self.big = np.abs(self.s)
        self.e = np.zeros(self.s.shape[:2])

    def copy(self):
        new = Bounds(self.s)
        new.big, new.e = self.big.copy(), self.e.copy()
        return new

    def token(self, k, v, g, beta):
        """One token; returns u [H, Dv] and how far it may be off."""
        Dk = k.shape[-1]
        a = np.exp(g.astype(np.float64))[:, None]
        beta = beta.astype(np.float64)[:, None]
        kk = (k ** 2).sum(-1)[:, None]
        kn = np.sqrt(kk)
        size = a * np.sqrt((self.big ** 2).sum(-1))
        self.s *= a[..., None]
        sk = (self.s * k[:, None]).sum(-1)
        u = beta * (v - sk)
        near = (Dk + 80) * U * (np.abs(beta) * (np.abs(v) + size * kn) + np.abs(u))
        eu = np.abs(beta) * kn * a * self.e + near
        self.s += u[..., None] * k[:, None]
        self.big = a[..., None] * self.big + np.abs(u)[..., None] * np.abs(k)[:, None]
        self.e = a * self.e * np.maximum(1, np.abs(1 - beta * kk)) + near * kn + (Dk + 80) * U * size
        return u, eu

    def read(self, q, scale, rounded):
        """o [H, Dv] and its bound; `rounded`: the relative rounding of the factors of o alone (2^-11 for f16)."""
        o = (self.s * q[:, None]).sum(-1)
        size = (self.big * np.abs(q)[:, None]).sum(-1)
        Dk = q.shape[-1]
        return scale * o, abs(scale) * (np.sqrt((q ** 2).sum(-1))[:, None] * self.e + (3 * rounded + (Dk + 80) * U) * size)


def used(src, slots):
    return -1 <= src < slots


def slot_written(src, dst, slots, b):
    to = dst[b]
    if not (0 <= to < slots and used(src[b], slots)):
        return -1
    for i in range(len(src)):
        if i != b and used(src[i], slots) and (src[i] == to or (i < b and dst[i] == to)):
            return -1
    return to


def _count(counts, b, M):
    return M if counts is None else max(0, min(M, int(counts[b])))


def _rows(q, k, v, g, beta, eps):
    H = v.shape[2]
    rep = lambda x: np.repeat(normalised(x, eps), H // x.shape[2], axis=2)  # noqa: E731
    return rep(q), rep(k), v.astype(np.float64)


def chain(q, k, v, g, beta, states, src, dst, counts=None, scale=None, eps=None, rounded=0.0):
    """(out, its bound, states after, their bound [S, H, Dv] in 2-norm of a row, their big); q, k [B, M, Hk, Dk]."""
    B, M, Hk, Dk = k.shape
    S = states.shape[0]
    scale = 1 / np.sqrt(Dk) if scale is None else scale
    out, tol = np.zeros(v.shape), np.zeros(v.shape)
    after, off = states.astype(np.float64).copy(), np.zeros(states.shape[:3])
    big = np.abs(after)
    for b in range(B):
        if not used(src[b], S):
            continue
        n = _count(counts, b, M)
        qs, ks, vs = _rows(q[b:b + 1, :n], k[b:b + 1, :n], v[b:b + 1, :n], g, beta, eps)
        st = Bounds(states[src[b]] if src[b] >= 0 else np.zeros_like(states[0]))
        for t in range(n):
            st.token(ks[0, t], vs[0, t], g[b, t], beta[b, t])
            out[b, t], tol[b, t] = st.read(qs[0, t], scale, rounded)
        to = slot_written(src, dst, S, b)
        if to >= 0:
            after[to], off[to], big[to] = st.s, st.e, st.big
    return out, tol, after, off, big


def tree(q, k, v, g, beta, states, src, parent, counts=None, scale=None, eps=None, rounded=0.0):
    """(out, its bound, keys, updates, their bound)."""
    B, M, Hk, Dk = k.shape
    scale = 1 / np.sqrt(Dk) if scale is None else scale
    out, tol, updates, utol = (np.zeros(v.shape) for _ in range(4))
    keys = np.zeros(k.shape)
    for b in range(B):
        if not used(src[b], states.shape[0]):
            continue
        n = _count(counts, b, M)
        qs, ks, vs = _rows(q[b:b + 1, :n], k[b:b + 1, :n], v[b:b + 1, :n], g, beta, eps)
        keys[b, :n] = normalised(k[b, :n], eps)
        begin, after = Bounds(states[src[b]] if src[b] >= 0 else np.zeros_like(states[0])), []
        for t in range(n):
            p = int(parent[b, t])
            st = (after[p] if 0 <= p < t else begin).copy()
            updates[b, t], utol[b, t] = st.token(ks[0, t], vs[0, t], g[b, t], beta[b, t])
            out[b, t], tol[b, t] = st.read(qs[0, t], scale, rounded)
            after.append(st)
    return out, tol, keys, updates, utol


def commit(states, keys, updates, g, result, src, dst):
    """(states [L, S, H, Dv, Dk] after, the sum of the sizes of what each value adds up)."""
    L, S, H = states.shape[:3]
    B, M, Hk = keys.shape[1:4]
    after, size = states.astype(np.float64).copy(), np.abs(states.astype(np.float64))
    for b in range(B):
        to = slot_written(src, dst, S, b)
        if to < 0:
            continue
        n = max(1, min(M, int(result[b, 1]) + 1))
        st = states[:, src[b]].astype(np.float64) if src[b] >= 0 else np.zeros_like(after[:, 0])
        big = np.abs(st)
        for i in range(n):
            t = 0 if i == 0 else int(result[b, 2 + i])
            if not 0 <= t < M:
                continue
            a = np.exp(g[:, b, t].astype(np.float64))[..., None, None]
            kt = np.repeat(keys[:, b, t].astype(np.float64), H // Hk, axis=1)[:, :, None]
            ut = updates[:, b, t].astype(np.float64)[..., None]
            st = a * st + ut * kt
            big = a * big + np.abs(ut) * np.abs(kt)
        after[:, to], size[:, to] = st, big
    return after, size
