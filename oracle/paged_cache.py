"""Oracle of the paged-cache operators — TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module: a plain transcription, in numpy and whole
numbers, of what include/cachegen.h says of cg_pages_* and
cg_attention_prefix_async.  A cache is a ``Cache`` of host arrays; every function
changes it in place and returns the status bits that it sets.  The attention is
computed in binary64, one query and head at a time, over the tokens of the row's
own table; the pools are read through float64.
"""
from __future__ import annotations

import dataclasses

import numpy as np

BAD_PAGE, REFUSED, NO_PAGES = 2, 4, 8


@dataclasses.dataclass
class Cache:
    k: np.ndarray       # fp16 [L][N][P][C]
    v: np.ndarray
    tables: np.ndarray  # int32 [R][B]
    lens: np.ndarray    # int32 [R]
    refs: np.ndarray    # int32 [N]

    @property
    def P(self):
        return self.k.shape[2]

    @property
    def N(self):
        return self.k.shape[1]

    def copy(self):
        return Cache(*(x.copy() for x in (self.k, self.v, self.tables, self.lens, self.refs)))


def empty(layers, pages, page_tokens, channels, rows, max_blocks, fill=0x7E5A):
    shape = (layers, pages, page_tokens, channels)
    return Cache(np.full(shape, fill, np.uint16).view(np.float16),
                 np.full(shape, fill, np.uint16).view(np.float16),
                 np.full((rows, max_blocks), -1, np.int32), np.zeros(rows, np.int32),
                 np.zeros(pages, np.int32))


def blocks(c: Cache, n):
    return -(-int(n) // c.P)


def row_ok(c, r):
    return 0 <= r < len(c.lens)


def len_ok(c, n):
    return 0 <= n <= c.tables.shape[1] * c.P


def copy(c: Cache, src, dst):
    status, todo = 0, []
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (0 <= s < c.N and 0 <= d < c.N):
            status |= BAD_PAGE
        elif s in list(dst) or list(dst).count(d) > 1:
            status |= REFUSED
        else:
            todo.append((s, d))
    for s, d in todo:
        c.k[:, d], c.v[:, d] = c.k[:, s], c.v[:, s]
    return status


def reserve(c: Cache, rows, starts, n_tokens):
    """Returns (status, slots)."""
    status, slots = 0, np.full(n_tokens, -1, np.int64)
    free = [p for p in range(c.N) if c.refs[p] == 0]
    used, short = 0, False
    plan = []
    for i, r in enumerate(rows):
        a, b = int(starts[i]), int(starts[i + 1])
        if (not row_ok(c, r) or list(rows).count(r) > 1 or not 0 <= a <= b <= n_tokens
                or not len_ok(c, c.lens[r]) or not len_ok(c, int(c.lens[r]) + b - a)):
            status |= REFUSED
            continue
        need = blocks(c, c.lens[r] + b - a) - blocks(c, c.lens[r])
        used += need
        if need and used > len(free):
            status |= NO_PAGES
            continue
        plan.append((r, a, b, free[used - need:used]))
    for r, a, b, pages in plan:
        n = int(c.lens[r])
        nb = blocks(c, n)
        c.tables[r, nb:nb + len(pages)] = pages
        c.refs[pages] = 1
        c.lens[r] = n + b - a
        for t in range(a, b):
            pos = n + t - a
            p = c.tables[r, pos // c.P]
            if 0 <= p < c.N:
                slots[t] = int(p) * c.P + pos % c.P
            else:
                status |= BAD_PAGE
    return status, slots


def write(c: Cache, layer0, slots, k_new, v_new):
    status = 0
    for t, s in enumerate(slots):
        if 0 <= s < c.N * c.P:
            for pool, new in ((c.k, k_new), (c.v, v_new)):
                pool[layer0:layer0 + new.shape[0], s // c.P, s % c.P] = new[:, t]
        elif s != -1:
            status |= BAD_PAGE
    return status


def fork(c: Cache, parents, children):
    status, plan = 0, []
    free = [p for p in range(c.N) if c.refs[p] == 0]
    used = 0
    for a, b in zip(parents, children):
        if (not row_ok(c, a) or not row_ok(c, b) or list(children).count(b) > 1
                or b in list(parents) or c.lens[b] != 0 or not len_ok(c, c.lens[a])):
            status |= REFUSED
            continue
        n, fresh = int(c.lens[a]), -1
        if n % c.P:
            if not 0 <= c.tables[a, blocks(c, n) - 1] < c.N:
                status |= BAD_PAGE
                continue
            used += 1
            if used > len(free):
                status |= NO_PAGES
                continue
            fresh = free[used - 1]
        plan.append((a, b, n, fresh))
    for a, b, n, fresh in plan:
        nb = blocks(c, n)
        c.tables[b, :nb] = c.tables[a, :nb]
        c.lens[b] = n
        for p in c.tables[a, :n // c.P]:
            if 0 <= p < c.N:
                c.refs[p] += 1
            else:
                status |= BAD_PAGE
        if fresh >= 0:
            old = c.tables[a, nb - 1]
            c.tables[b, nb - 1] = fresh
            c.refs[fresh] = 1
            for pool in (c.k, c.v):
                pool[:, fresh, :n % c.P] = pool[:, old, :n % c.P]
    return status


def free(c: Cache, rows):
    status, done = 0, set()
    for r in rows:
        if r in done or not row_ok(c, r) or not len_ok(c, c.lens[r]):
            status |= REFUSED
            continue
        done.add(r)
        for b in range(blocks(c, c.lens[r])):
            p = c.tables[r, b]
            c.tables[r, b] = -1
            if not 0 <= p < c.N:
                status |= BAD_PAGE
            elif c.refs[p] <= 0:
                status |= REFUSED
            else:
                c.refs[p] -= 1
        c.lens[r] = 0
    return status


def compact(c: Cache):
    """Returns (status, number of pages in use)."""
    live = int((c.refs > 0).sum())
    src = [p for p in range(live, c.N) if c.refs[p] > 0]
    dst = [p for p in range(live) if c.refs[p] == 0]
    status = 0 if len(src) == len(dst) else REFUSED
    to = dict(zip(src, dst))
    for a, b in to.items():
        c.k[:, b], c.v[:, b] = c.k[:, a], c.v[:, a]
        c.refs[b], c.refs[a] = c.refs[a], 0
    for r, n in enumerate(c.lens):
        if len_ok(c, n):
            for b in range(blocks(c, n)):
                c.tables[r, b] = to.get(int(c.tables[r, b]), c.tables[r, b])
    return status, live


def attention(c: Cache, layer, q, scale, rows, q_starts, group_starts=None, prefix_lens=None):
    """Returns (status, {query: [H] records}) with a record per query and head:
    out (binary64 [d]), lse, mean_abs = sum p |v| (binary64 [d]), size = the largest
    scale * sum |q k| of the row, tokens.  Queries of no sequence have no record."""
    n_q, H, d = q.shape
    C = c.k.shape[3]
    kv = C // d
    G = H // kv
    status, got = 0, {}
    n_seqs = len(q_starts) - 1
    for s in range(n_seqs):
        row = s if rows is None else int(rows[s])
        a, b = int(q_starts[s]), int(q_starts[s + 1])
        if a >= b:
            continue
        ok = row_ok(c, row) and len_ok(c, c.lens[row]) and 0 <= a and b <= n_q
        n = int(c.lens[row]) if ok else 0
        pre, first = 0, row
        for g in range(0 if group_starts is None else len(group_starts) - 1):
            if group_starts[g] <= s < group_starts[g + 1]:
                pre = int(prefix_lens[g])
                f = int(group_starts[g])
                first = f if rows is None else int(rows[f])
        if pre < 0 or (pre > 0 and (pre + b - a > n or not row_ok(c, first) or not len_ok(c, c.lens[first])
                                    or c.lens[first] < pre)):
            ok = False
        if not ok:
            status |= REFUSED
        for j in range(a, b):
            lim = max(0, n - (b - a) + (j - a) + 1) if ok else 0
            t = np.arange(lim)
            page = np.where(t < pre, c.tables[first, t // c.P], c.tables[row, t // c.P]) if lim else t
            inside = (page >= 0) & (page < c.N)
            if not inside.all():
                status |= BAD_PAGE
            page, t = page[inside], t[inside]
            K = c.k[layer, page, t % c.P].astype(np.float64).reshape(len(t), kv, d)
            V = c.v[layer, page, t % c.P].astype(np.float64).reshape(len(t), kv, d)
            recs = []
            for h in range(H):
                x = q[j, h].astype(np.float64)
                with np.errstate(invalid="ignore"):
                    sc = scale * (K[:, h // G] @ x)
                    m = sc.max() if len(t) else -np.inf
                    if m == -np.inf:
                        recs.append(dict(out=np.zeros(d), lse=-np.inf, mean_abs=np.zeros(d), size=0.0,
                                         tokens=0, vmax=0.0, l=1.0))
                        continue
                    e = np.exp(sc - m)
                    l = e.sum()
                    p = e / l
                    recs.append(dict(out=p @ V[:, h // G], lse=m + np.log(l),
                                     mean_abs=p @ np.abs(V[:, h // G]),
                                     size=abs(scale) * (np.abs(K[:, h // G]) @ np.abs(x)).max(),
                                     tokens=len(t), vmax=np.abs(V[:, h // G]).max(), l=l))
            got[j] = recs
    return status, got
