"""Plain 64-bit forms of the key/value-cache operators, for the tests: loops over
sequences, heads and rows on the CPU, sharing no code with the CUDA path.

A `State` holds a cache on the CPU the way its operators see it: per sequence
and kv-head a list of (key, value, position, weight), in slot order. `make`
lays one out in pages in a drawn order, with NaN in every place that no key
holds and wild page ids where the table is not read.
"""
from __future__ import annotations

import math
from dataclasses import dataclass, field
from typing import List, Optional

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# half a step of the type, relative to the value
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@dataclass
class Layout:
    """A cache's tensors, on the CPU."""
    k: torch.Tensor           # [n_pages, page, h_kv, d]
    v: torch.Tensor
    table: Optional[torch.Tensor]
    lengths: torch.Tensor
    next_pos: Optional[torch.Tensor]
    positions: Optional[torch.Tensor]
    weights: Optional[torch.Tensor]
    real: List[List[int]] = field(default_factory=list)   # page ids of each sequence

    def clone(self):
        c = lambda t: None if t is None else t.clone()  # noqa: E731
        return Layout(*[c(getattr(self, f)) for f in ("k", "v", "table", "lengths", "next_pos", "positions", "weights")],
                      real=self.real)

    @property
    def cap(self):
        return (self.table.shape[1] if self.table is not None else 1) * self.k.shape[1]

    def where(self, i, slots):
        page = self.k.shape[1]
        ids = np.asarray(self.real[i], dtype=np.int64)
        return ids[np.asarray(slots) // page], np.asarray(slots) % page

    def rows(self, i, g, n):
        pg, at = self.where(i, np.arange(n))
        return self.k[pg, at, g], self.v[pg, at, g]

    def pos(self, i, g, n):
        return self.positions[i, g, :n].numpy().astype(np.int64) if self.positions is not None else np.arange(n)

    def next(self, i):
        return int(self.next_pos[i]) if self.next_pos is not None else int(self.lengths[i])


def make(seed, lens, h_kv, d, dtype, page, *, room=0, tracked=False, evicted=False, spare=2, wild=True):
    """Sequences of these lengths with room for `room` more keys; page 0: one
    run of slots each. `tracked`: with positions and weights; `evicted`: with
    positions as earlier evictions leave them (gaps, another order per head)."""
    g = torch.Generator().manual_seed(seed)
    rs = np.random.RandomState(seed)
    b, dt = len(lens), DT[dtype]
    most = max([n + room for n in lens] + [1])
    psz = page or most
    per = -(-most // psz)
    n_pages = b * per + spare
    k = torch.full((n_pages, psz, h_kv, d), math.nan, dtype=dt)
    v = torch.full((n_pages, psz, h_kv, d), math.nan, dtype=dt)
    if page:
        ids = rs.permutation(n_pages)[:b * per].reshape(b, per)
    else:
        ids = np.arange(b).reshape(b, 1)
    table = torch.from_numpy(ids.astype(np.int32)) if page else None
    lay = Layout(k, v, table, torch.tensor(lens, dtype=torch.int32), None, None, None, ids.tolist())
    for i, n in enumerate(lens):
        pg, at = lay.where(i, np.arange(n))
        k[pg, at] = torch.randn(n, h_kv, d, generator=g).to(dt)
        v[pg, at] = torch.randn(n, h_kv, d, generator=g).to(dt)
        if page and wild:
            used = -(-(n + room) // psz)
            table[i, used:] = torch.tensor(rs.choice([-1, -7, n_pages, 2 ** 31 - 1], per - used), dtype=torch.int32)
    if tracked or evicted:
        lay.positions = torch.full((b, h_kv, lay.cap), -5, dtype=torch.int32)
        lay.weights = torch.full((b, h_kv, lay.cap), math.nan)
        lay.next_pos = torch.zeros(b, dtype=torch.int32)
        for i, n in enumerate(lens):
            pos = np.cumsum(rs.randint(1, 4, n)) - 1 if evicted else np.arange(n)
            lay.next_pos[i] = int(pos[-1]) + 1 if n else 0
            for h in range(h_kv):
                p = rs.permutation(pos) if evicted else pos
                lay.positions[i, h, :n] = torch.from_numpy(p.astype(np.int32))
                w = np.floor(np.exp(2 * rs.randn(n)) * 16) / 16
                lay.weights[i, h, :n] = torch.from_numpy(w.astype(np.float32))
    return lay


def chain(t):
    return [(1 << (r + 1)) - 1 for r in range(t)]


def tree_masks(seed, b, t, empty=0.0):
    """Ancestor masks of drawn trees (forests too); `empty`: share of padding rows."""
    rs = np.random.RandomState(seed)
    out = np.zeros((b, t), dtype=np.uint64)
    for i in range(b):
        for r in range(t):
            if rs.rand() < empty:
                continue
            up = rs.randint(-1, r) if r else -1
            m = int(out[i, up]) if up >= 0 else 0
            out[i, r] = np.uint64(m | (1 << r))
    return torch.from_numpy(out.view(np.int64).copy())


@dataclass
class Forward:
    o: torch.Tensor       # [b, t, h_q, d] float64
    lse: torch.Tensor     # [b, h_q, t]
    tol_o: torch.Tensor
    tol_lse: torch.Tensor


def score_error(q, k, scale, d):
    """Bound on the error of a score (natural units) formed in fp32 from 16-bit
    inputs: d products of exact value summed with an error of at most one fp32
    step (2^-23; matrix units may truncate) of the partial sum each, and the
    scale, its log2(e) multiple and the subtraction rounded."""
    mag = (q.abs() @ k.abs().T) * scale
    return mag * (d + 8) * 2.0 ** -23


def forward(lay, q, k, v, *, scale, window=-1, tree=None, q_lens=None, sink=None, dtype="bf16"):
    b, t, h_q, d = q.shape
    h_kv = k.shape[2]
    grp = h_q // h_kv
    f64 = torch.float64
    o = torch.zeros(b, t, h_q, d, dtype=f64)
    lse = torch.full((b, h_q, t), -math.inf, dtype=f64)
    tol_o, tol_l = torch.zeros(b, t, h_q, d, dtype=f64), torch.zeros(b, h_q, t, dtype=f64)
    u = U[dtype]
    for i in range(b):
        n, nq = int(lay.lengths[i]), t if q_lens is None else int(q_lens[i])
        line = chain(t) if tree is None else [int(x) % 2 ** 64 for x in tree[i].tolist()]
        line = [x & ((1 << nq) - 1) for x in line]
        deep = [bin(x).count("1") - 1 for x in line]
        for r in range(nq):
            for h in range(h_q):
                g = h // grp
                ks, vs = lay.rows(i, g, n)
                pos = lay.next(i) + deep[r]
                see = np.ones(n, bool) if window < 0 else pos - lay.pos(i, g, n) <= window
                own = [x for x in range(nq) if line[r] >> x & 1 and (window < 0 or deep[r] - deep[x] <= window)]
                if not line[r] >> r & 1:
                    see, own = np.zeros(n, bool), []
                kk = torch.cat([ks[see], k[i, own, g]]).to(f64)
                vv = torch.cat([vs[see], v[i, own, g]]).to(f64)
                qq = q[i, r, h].to(f64)[None]
                s = (qq @ kk.T * scale)[0]
                z = torch.logsumexp(s, 0) if len(s) else torch.tensor(-math.inf, dtype=f64)
                if sink is not None:
                    z = torch.logaddexp(z, sink[h].to(f64))
                lse[i, h, r] = z
                if not len(s):
                    continue
                p = torch.exp(s - z)
                o[i, r, h] = p @ vv
                # scores off by es: p and the sum off by a factor e^es each; the exponentials
                # within 2^-21, the sums of m terms within m steps
                m = len(s) + 8
                es = float(score_error(qq, kk, scale, d).max()) + float(s.abs().max()) * 2.0 ** -22
                rel = 2 * es + 2.0 ** -20 + m * 2.0 ** -23
                tol_l[i, h, r] = es + 2.0 ** -20 + m * 2.0 ** -23 + abs(float(z)) * 2.0 ** -22
                # O in 16 bits; P in 16 bits (f16's smallest step besides, relative to the largest p)
                tol_o[i, r, h] = (u * o[i, r, h].abs() + (u + rel) * (1 + u) * (p @ vv.abs()) +
                                  (2.0 ** -25 * m * float(p.max()) * float(vv.abs().max()) if dtype == "f16" else 0) + 2.0 ** -24)
    return Forward(o, lse, tol_o, tol_l)


def weigh(lay, q, lse, *, scale, window=-1, q_pos=None):
    """The weights after the call, and how far off they may be."""
    b, t, h_q, d = q.shape
    h_kv = lay.k.shape[2]
    grp = h_q // h_kv
    w = lay.weights.double().clone()
    tol = w.abs() * 2.0 ** -24
    for i in range(b):
        n = int(lay.lengths[i])
        for g in range(h_kv):
            ks = lay.rows(i, g, n)[0].double()
            pos = torch.from_numpy(lay.pos(i, g, n))
            add = torch.zeros(n, dtype=torch.float64)
            off = torch.zeros(n, dtype=torch.float64)
            for r in range(t):
                p = lay.next(i) - t + r if q_pos is None else int(q_pos[i, r])
                if p < 0:
                    continue
                see = pos <= p
                if window >= 0:
                    see = see & (p - pos <= window)
                for h in range(g * grp, (g + 1) * grp):
                    z = float(lse[i, h, r])
                    if not math.isfinite(z):
                        continue
                    qq = q[i, r, h].double()[None]
                    s = (qq @ ks.T * scale)[0]
                    es = score_error(qq, ks, scale, d)[0] + (s.abs() + abs(z)) * 2.0 ** -22 + 2.0 ** -20
                    e = torch.where(see, torch.exp(s - z), torch.zeros_like(s))
                    add += e
                    off += e * es
            w[i, g, :n] += add
            tol[i, g, :n] += off * 1.01 + (add + w[i, g, :n].abs()) * (t * grp + 2) * 2.0 ** -23
    return w, tol


def append(lay, k, v, *, index=None, counts=None, offsets=None, skip=()):
    """The cache after the call (a new Layout); `skip`: sequences left alone."""
    out = lay.clone()
    for i in range(len(lay.lengths)):
        if i in skip:
            continue
        if offsets is not None:
            src = list(range(int(offsets[i]), int(offsets[i + 1])))
        else:
            src = index[i].tolist() if index is not None else list(range(k.shape[1]))
        if counts is not None:
            src = src[:int(counts[i])]
        n = int(lay.lengths[i])
        slots = np.arange(n, n + len(src))
        pg, at = lay.where(i, slots)
        out.k[pg, at] = k[src] if offsets is not None else k[i, src]
        out.v[pg, at] = v[src] if offsets is not None else v[i, src]
        out.lengths[i] = n + len(src)
        if lay.positions is not None:
            out.positions[i, :, n:n + len(src)] = torch.arange(len(src), dtype=torch.int32) + lay.next_pos[i]
            out.next_pos[i] += len(src)
        if lay.weights is not None:
            out.weights[i, :, n:n + len(src)] = 0
    return out


def evict(lay, keep, first, recent):
    out = lay.clone()
    for i in range(len(lay.lengths)):
        n = int(lay.lengths[i])
        if n <= keep:
            continue
        out.lengths[i] = keep
        for g in range(lay.k.shape[2]):
            def order(j):
                p, w = int(lay.positions[i, g, j]), float(lay.weights[i, g, j])
                if p < first or p >= int(lay.next_pos[i]) - recent:
                    return (0, 0.0, j)
                return (1, 0.0, j) if math.isnan(w) else (2, -w, j)
            stay = set(sorted(range(n), key=order)[:keep])
            free = [j for j in range(min(n, keep)) if j not in stay]
            come = [j for j in range(keep, n) if j in stay]
            assert len(free) == len(come)
            if free:
                (sp, sa), (dp, da) = lay.where(i, come), lay.where(i, free)
                out.k[dp, da, g] = lay.k[sp, sa, g]
                out.v[dp, da, g] = lay.v[sp, sa, g]
                out.positions[i, g, free] = lay.positions[i, g, come]
                out.weights[i, g, free] = lay.weights[i, g, come]
    return out
