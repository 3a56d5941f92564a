"""Beam search around the cache: selection of candidates, forks of the block
tables.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

* ``beam_select``: candidates as float64 values, sorted by value and index.
* ``fork_tables``: "19.2 KV Cache 系统化管理" §19.2.2 (写时复制: forks share blocks,
  a writer copies a shared one) as a simulation with one reference count per
  block and a queue of free ones.

Pinned in ``tests/test_oracle_beam_pins.py``.
"""

from __future__ import annotations

import math
from collections import Counter, deque

import numpy as np

__all__ = ["beam_select", "fork_tables"]


def beam_select(logits, scores, num_select, finished=None, eos=-1):
    """``logits`` float64 [R * B, V], ``scores`` [R, B] -> (tokens, parents,
    scores, finished), each [R, num_select]."""
    R, B = scores.shape
    V = logits.shape[1]
    tokens = np.full((R, num_select), -1, np.int32)
    parents = np.full((R, num_select), -1, np.int32)
    best = np.full((R, num_select), -np.inf)
    over = np.ones((R, num_select), bool)
    for r in range(R):
        found = []
        for b in range(B):
            if finished is not None and finished[r, b]:
                found.append((-float(scores[r, b]), b, eos))
                continue
            x = np.asarray(logits[r * B + b], np.float64)
            if np.isnan(x).any() or (x == np.inf).any():
                continue
            m = x.max()
            if m == -np.inf:
                continue
            lse = m + math.log(math.fsum(np.exp(x - m)))
            c = float(scores[r, b]) + x - lse
            order = np.lexsort((np.arange(V), -c))[:num_select]
            found += [(-c[v], b, int(v)) for v in order]
        found = sorted(f for f in found if math.isfinite(f[0]))[:num_select]
        for n, (c, b, v) in enumerate(found):
            tokens[r, n], parents[r, n], best[r, n] = v, b, -c
            over[r, n] = v == eos or (finished is not None and bool(finished[r, b]))
    return tokens, parents, best, over


def fork_tables(parents, lens, held, shared, tables, ring, state, K, out_tables=None):
    """Returns a dict of the outputs; ``tables`` [R * B, width]; ``out_tables``:
    what the table rows hold where nothing is written (default: ``tables``)."""
    R, B = parents.shape
    S, width = tables.shape
    size = len(ring)
    head, tail = int(state[0]), int(state[1])
    lens, held = [int(x) for x in lens], [int(x) for x in held]
    shared = [0] * S if shared is None else [int(x) for x in shared]
    new = np.array(tables if out_tables is None else out_tables)
    ring = np.array(ring)
    same = dict(lens=lens, held=held, state=[head, tail], ring=ring, pairs=[[-1, -1]] * S)
    bad_groups = set()
    for s in range(S):
        p = int(parents[s // B, s % B])
        if not -1 <= p < B or lens[s] < 0 or not 0 <= held[s] <= width or shared[s] < 0 \
                or lens[s] > held[s] * K:
            bad_groups.add(s // B)
    free = deque(int(ring[i % size]) for i in range(head, min(tail, head + size))) \
        if 0 <= head <= tail else deque()
    enough = len(free)
    live = sum(int(p >= 0) for p in parents.flatten())
    rows, lens2, held2, pairs, taken, given = [], [], [], [], 0, []
    count = Counter()                     # rows that list a block, over the whole pool
    for s in range(S):
        if s // B not in bad_groups:
            count.update(int(x) for x in tables[s, :held[s]])
    for g in range(R):
        if g in bad_groups:
            rows += [[]] * B
            continue
        used = set()
        old = [list(map(int, tables[g * B + b, :held[g * B + b]])) for b in range(B)]
        for i in range(B):
            p = int(parents[g, i])
            if p < 0:
                rows.append([]), lens2.append(0), held2.append(0), pairs.append([-1, -1])
                continue
            n = lens[g * B + p]
            row = list(old[p])
            pair = [-1, -1]
            if p in used:
                row = row[:-(-n // K)]
                if n % K:
                    taken += 1
                    block = free.popleft() if free else -99
                    pair = [row[n // K], block]
                    row[n // K] = block
            used.add(p)
            count.update(row)
            rows.append(row), lens2.append(n), held2.append(len(row)), pairs.append(pair)
        for b in range(B):
            count.subtract(old[b])
        for c in range(max(held[g * B:g * B + B], default=0)):
            for b in range(B):
                if shared[g * B + b] <= c < len(old[b]) and count[old[b][c]] == 0 \
                        and old[b][c] not in given:
                    given.append(old[b][c])
    code = 0
    if bad_groups or not 0 <= tail - head <= size or head < 0 or tail + len(given) - head > size:
        code = 3
    elif taken > enough:
        code = 1
    totals = [code, live, taken, len(given)]
    if code:
        if out_tables is not None:
            for s in range(S):
                h = max(0, min(held[s], width))
                new[s, :h] = tables[s, :h]
        return dict(same, tables=new, totals=totals)
    for s in range(S):
        new[s, :len(rows[s])] = rows[s]
    for i, x in enumerate(given):
        ring[(tail + i) % size] = x
    return dict(tables=new, lens=lens2, held=held2, state=[head + taken, tail + len(given)],
                ring=ring, pairs=pairs, totals=totals)
