"""Plain 64-bit definitions of the paged-cache operators, for the tests: page
bookkeeping as sequential Python over lists, rotary positions and attention
in float64 on the CPU. They share nothing with the library."""
import math

import torch

BAD_PAGE, CAPACITY = 8, 2


class Pages:
    """Page state on the host. `pool` is a uint8 tensor [ranks, pages, bytes]."""

    def __init__(self, tables, lens, refs, pool, page_tokens):
        self.tables = [list(r) for r in tables]
        self.lens, self.refs = list(lens), list(refs)
        self.pool, self.bt = pool.clone(), page_tokens
        self.status = 0

    def _need(self, n):
        return -(-n // self.bt)

    def _first(self, seqs):
        """Indices of the requests that count: in range, the first of their sequence."""
        seen, good = set(), []
        for i, s in enumerate(seqs):
            if 0 <= s < len(self.lens) and s not in seen:
                seen.add(s)
                good.append(i)
            else:
                self.status |= BAD_PAGE
        return good

    def extend(self, seqs, add):
        cap = len(self.tables[0]) * self.bt
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        used = 0
        for i in self._first(seqs):
            s, n = seqs[i], add[i]
            if n < 0 or not 0 <= self.lens[s] <= cap or self.lens[s] + n > cap:
                self.status |= BAD_PAGE
                continue
            have = self._need(self.lens[s])
            need = self._need(self.lens[s] + n) - have
            take = free[used:used + need]
            used += need
            if need and used > len(free):
                self.status |= CAPACITY
                continue
            for k, p in enumerate(take):
                self.tables[s][have + k] = p
                self.refs[p] = 1
            self.lens[s] += n

    def fork(self, parents, children):
        cap = len(self.tables[0]) * self.bt
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        lens, tables = list(self.lens), [list(r) for r in self.tables]
        pool, used = self.pool.clone(), 0
        for i in self._first(children):
            c, p = children[i], parents[i]
            if not 0 <= p < len(lens) or lens[c] != 0 or not 0 <= lens[p] <= cap:
                self.status |= BAD_PAGE
                continue
            full, part = divmod(lens[p], self.bt)
            page = None
            if part:
                used += 1
                if used > len(free):
                    self.status |= CAPACITY
                    continue
                page = free[used - 1]
            row = [-1] * len(tables[0])
            for k in range(full):
                row[k] = tables[p][k]
                if 0 <= row[k] < len(self.refs):
                    self.refs[row[k]] += 1
                else:
                    self.status |= BAD_PAGE
            if part:
                row[full] = page
                self.refs[page] = 1
                src = tables[p][full]
                if 0 <= src < len(self.refs):
                    self.pool[:, page] = pool[:, src]
                else:
                    self.status |= BAD_PAGE
            self.tables[c], self.lens[c] = row, lens[p]

    def free(self, seqs):
        cap = len(self.tables[0]) * self.bt
        for i in self._first(seqs):
            s = seqs[i]
            if not 0 <= self.lens[s] <= cap:
                self.status |= BAD_PAGE
            n = min(self._need(max(self.lens[s], 0)), len(self.tables[s]))
            for p in self.tables[s][:n]:
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.status |= BAD_PAGE
            self.tables[s], self.lens[s] = [-1] * len(self.tables[s]), 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] <= 0]
        to = dict(zip(movers, holes))
        for p, h in to.items():
            self.pool[:, h] = self.pool[:, p]
            self.refs[h], self.refs[p] = self.refs[p], 0
        for s, n in enumerate(self.lens):
            n = min(self._need(max(n, 0)), len(self.tables[s]))
            for k in range(n):
                p = self.tables[s][k]
                if not 0 <= p < len(self.refs):
                    self.status |= BAD_PAGE
                self.tables[s][k] = to.get(p, p)
        return live, to

    def copy(self, src, dst):
        n = len(self.refs)
        ok = [0 <= s < n and 0 <= d < n for s, d in zip(src, dst)]
        writer = {}
        for i, (s, d) in enumerate(zip(src, dst)):
            if ok[i] and s != d:
                writer.setdefault(d, i)
        pool = self.pool.clone()
        for i, (s, d) in enumerate(zip(src, dst)):
            if ok[i] and s == d:
                continue
            if not ok[i] or writer[d] != i or s in writer:
                self.status |= BAD_PAGE
                continue
            self.pool[:, d] = pool[:, s]


def rows_of(lens, q_off):
    """(sequence, position) of every row that belongs to one."""
    return [(b, lens[b] - (hi - lo) + j) for b, (lo, hi) in enumerate(zip(q_off, q_off[1:]))
            for j in range(hi - lo)]


def rotate(x, pos, inv_freq, rot, interleaved, mscale):
    """x [rows, heads, dim] float64, pos [rows]."""
    a = pos.double()[:, None] * inv_freq.double()
    c, s = (mscale * a.cos())[:, None], (mscale * a.sin())[:, None]
    y = x.clone()
    if interleaved:
        i, j = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        i, j = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def attend(q, k, v, sees, scale):
    """One sequence and KV head: q [rows, dim], k and v [keys, dim] float64, sees [rows, keys]
    bool. Returns out, lse, the mean of |v| under the weights, and the bound on |q||k| products
    that the score errors go by."""
    s = scale * (q @ k.t())
    s = torch.where(sees, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, 1)
    p = torch.where(sees, (s - lse[:, None]).exp(), torch.zeros_like(s))
    empty = ~sees.any(1)
    p[empty] = 0
    size = torch.where(sees, abs(scale) * (q.abs() @ k.abs().t()), torch.zeros_like(s))
    top = size.amax(1) if s.shape[1] else torch.zeros(len(q), dtype=torch.float64)
    return p @ v, lse, p @ v.abs(), top, p
