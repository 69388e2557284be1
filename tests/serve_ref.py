"""Plain implementations, in 64 bits or in whole numbers, of the serving
operators, and the bounds their results are held to.  Imported by tests only."""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24  # unit roundoff of fp32


# ------------------------------------------------------------------ attention

def attention(q, k, v, table, lens, prefix_pages=None, prefix_len=None, scale=None):
    """(out, lse, bound of out, bound of lse) in 64 bits on the CPU; rows of
    unused sequences are NaN.  Positions are visited one by one.

    The bounds count, for a row over n positions with s_j = scale q.k_j,
    S = scale sum |q||k| (largest over j) and A = sum_j p_j |v_j|:
      e_s  = (d + 2) u S + 4 u max |s|: a product sum of d terms in fp32, the
             scaling, and the exponent's rounding (scores in powers of two)
      e_p  = 2 e_s + 2^-21: the error of a weight and of the sum it is divided
             by, each with an exponential good to 2^-22
      out: A (e_p + h + (n + 8) u) + h |out| + the smallest subnormal step,
           h = half a step of the type (the weight's own rounding, then the
           output's)
      lse: e_s + (n + 8) u + 2^-21 + 4 u |lse|
    """
    B, T, nq, d = q.shape
    _, nkv, page, _ = k.shape
    G = nq // nkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    h = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
    qd = q.double().cpu()
    out = torch.full((B, T, nq, d), math.nan, dtype=torch.float64)
    lse = torch.full((B, T, nq), math.nan, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    table, lens = table.cpu(), lens.cpu().tolist()
    pre = int(prefix_len.item()) if prefix_pages is not None and prefix_pages.numel() else 0
    pp = prefix_pages.cpu() if pre else None
    for b in range(B):
        if lens[b] < 0:
            continue
        n = lens[b]
        where = [((int(pp[j // page]) if j < pre else int(table[b, j // page])), j % page) for j in range(n)]
        pg = torch.tensor([x for x, _ in where], dtype=torch.long, device=k.device)
        rw = torch.tensor([x for _, x in where], dtype=torch.long, device=k.device)
        kk = k[pg, :, rw].double().cpu() if n else torch.zeros(0, nkv, d, dtype=torch.float64)  # [n][kv head][d]
        vv = v[pg, :, rw].double().cpu() if n else torch.zeros(0, nkv, d, dtype=torch.float64)
        for t in range(T):
            m = max(0, n - (T - 1 - t))
            for hd in range(nq):
                if m == 0:
                    out[b, t, hd] = 0
                    lse[b, t, hd] = -math.inf
                    continue
                K, V, x = kk[:m, hd // G], vv[:m, hd // G], qd[b, t, hd]
                s = scale * (K @ x)
                S = float((abs(scale) * (K.abs() @ x.abs())).max())
                p = torch.softmax(s, 0)
                o = p @ V
                e_s = (d + 2) * U32 * S + 4 * U32 * float(s.abs().max())
                e_p = 2 * e_s + 2.0 ** -21
                out[b, t, hd] = o
                tol_o[b, t, hd] = (p @ V.abs()) * (e_p + h + (m + 8) * U32) + h * o.abs() + tiny
                z = torch.logsumexp(s, 0)
                lse[b, t, hd] = z
                tol_l[b, t, hd] = e_s + (m + 8) * U32 + 2.0 ** -21 + 4 * U32 * float(z.abs())
    return out, lse, tol_o, tol_l


def check_attention(got, want, what=""):
    """got: (out, lse) of the kernel; want: what attention() returns."""
    out, lse, tol_o, tol_l = want
    used = ~torch.isnan(lse)
    o, l = got[0].double().cpu(), got[1].double().cpu()
    err = (o - out).abs()
    bad = used[..., None] & ~((err <= tol_o))
    assert not bad.any(), f"{what}: out off by {float(err[bad].max())} (allowed {float(tol_o[bad].max())}) at {bad.nonzero()[0].tolist()}"
    empty = used & torch.isinf(lse)
    assert (l[empty] == -math.inf).all(), what
    full = used & ~empty
    err = (l - lse).abs()[full]
    assert (err <= tol_l[full]).all(), f"{what}: lse off by {float(err.max())}"


# ------------------------------------------------------------------ cache pages

class Pages:
    """A paged cache on the host: bookkeeping as Python lists, rows as numpy arrays [layers][pages][heads][page][d]."""

    def __init__(self, k, v, n_seqs, max_pages):
        self.k, self.v = k.copy(), v.copy()
        self.P, self.page, self.max_pages = k.shape[1], k.shape[3], max_pages
        self.len = [0] * n_seqs
        self.refs = [0] * self.P
        self.free = list(range(self.P - 1, -1, -1))
        self.held = [[] for _ in range(n_seqs)]
        self.error = 0

    def _fail(self, code):
        self.error = self.error or code

    def _rows(self, src, dst, n):
        for x in (self.k, self.v):
            x[:, dst, :, :n] = x[:, src, :, :n]

    def resize(self, seqs, lens, INPUT=-7, OOM=-8):
        todo, seen, given = [], set(), []
        cap = self.max_pages * self.page
        for s, n in zip(seqs, lens):
            if not (0 <= s < len(self.len) and 0 <= n <= cap) or s in seen:
                self._fail(INPUT)
            else:
                todo.append((s, n))
            seen.add(s)
        for s, n in todo:
            while len(self.held[s]) > -(-n // self.page):
                p = self.held[s].pop()
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    given.append(p)
        self.free += sorted(given)
        for s, n in todo:
            have = self.len[s]
            cow = n > have and have % self.page != 0 and self.refs[self.held[s][have // self.page]] > 1
            if n > have and cow + -(-n // self.page) - -(-have // self.page) > len(self.free):
                self._fail(OOM)
                continue
            if cow:
                old = self.held[s][have // self.page]
                new = self.free.pop()
                self.refs[old] -= 1
                self.refs[new] = 1
                self.held[s][have // self.page] = new
                self._rows(old, new, have % self.page)
            while len(self.held[s]) < -(-n // self.page):
                p = self.free.pop()
                self.refs[p] = 1
                self.held[s].append(p)
            self.len[s] = n

    def fork(self, parents, children, INPUT=-7, OOM=-8):
        before = [(n, list(h)) for n, h in zip(self.len, self.held)]
        used = set()
        for p, c in zip(parents, children):
            S = len(self.len)
            if not (0 <= p < S and 0 <= c < S) or p == c or before[c][0] != 0 or c in used:
                self._fail(INPUT)
                continue
            used.add(c)
            n, held = before[p]
            full, rem = divmod(n, self.page)
            if rem and not self.free:
                self._fail(OOM)
                continue
            self.held[c] = held[:full]
            for x in held[:full]:
                self.refs[x] += 1
            if rem:
                new = self.free.pop()
                self.refs[new] = 1
                self.held[c].append(new)
                self._rows(held[full], new, rem)
            self.len[c] = n

    def compact(self):
        live = [p for p in range(self.P) if self.refs[p] > 0]
        n = len(live)
        move = dict(zip([p for p in live if p >= n], [p for p in range(n) if self.refs[p] == 0]))
        for a, b in move.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self._rows(a, b, self.page)
        self.held = [[move.get(p, p) for p in h] for h in self.held]
        self.free = list(range(self.P - 1, n - 1, -1))

    def check(self, state, k=None, v=None):
        """Every word of a KvState that has a meaning, and the pools."""
        assert int(state.n_free) == len(self.free)
        buf = state.buffer.cpu().numpy()
        S, P = len(self.len), self.P
        np.testing.assert_array_equal(buf[4:4 + S], self.len)
        np.testing.assert_array_equal(buf[4 + S:4 + S + P], self.refs)
        np.testing.assert_array_equal(buf[4 + S + P:4 + S + P + len(self.free)], self.free)
        table = np.full((S, self.max_pages), -1)
        for s, h in enumerate(self.held):
            table[s, :len(h)] = h
        np.testing.assert_array_equal(buf[4 + S + 2 * P:].reshape(S, -1), table)
        if k is not None:
            assert np.array_equal(k, self.k) and np.array_equal(v, self.v), "rows"


# ------------------------------------------------------------------ sampling

def probs(z, t):
    """Softmax of one row in 64 bits; zeros where there is no distribution."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max() if z.size else -np.inf
    if np.isnan(z).any() or not np.isfinite(m) or not (0 <= t < np.inf):
        return np.zeros_like(z)
    if t == 0:
        p = np.zeros_like(z)
        p[int(np.argmax(z))] = 1
        return p
    e = np.exp((z - m) / np.float64(t))
    return e / e.sum()


def verify(p, q, x, n, u):
    """(tokens that stand, the token after them or -1) of one sequence; p [n + 1][V], q [n][V] or None."""
    def pos(a):
        a = np.asarray(a, dtype=np.float64)
        return np.where((a > 0) & np.isfinite(a), a, 0.0)

    V = p.shape[1]
    a = 0
    while a < n and 0 <= x[a] < V:
        qx = pos(q[a][x[a]]) if q is not None else 1.0
        if not float(u[a]) * qx < pos(p[a][x[a]]):
            break
        a += 1
    r = pos(p[a])
    if a < n:
        if q is not None:
            less = np.maximum(r - pos(q[a]), 0)
        else:
            less = r.copy()
            if 0 <= x[a] < V:
                less[x[a]] = 0
        r = less if less.any() else r
    if not r.any():
        return a, -1
    c = np.cumsum(r)
    return a, int(np.argmax(c > float(u[len(u) - 1]) * c[-1]))
