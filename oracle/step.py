"""One engine step around the attention: block tables from lengths, head
norms + rotation, verification of drafted tokens.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

* ``step_tables``: "19.2 KV Cache 系统化管理" §19.2.2 (a request gets a new
  block when its last one is full) and "推理与 KV Cache 02", 从一个位置找到缓存块
  (slot = block * K + offset), as a plain simulation with a queue of free
  blocks.
* ``norm_rope``: RMS norm of one head row and the rotation of its pairs, in
  float64.
* ``verify``: acceptance of drafted tokens and the draw of the next one, in
  Python integers (the draw counts every weight in units of 2^-40, so it is
  exact).

Pinned in ``tests/test_oracle_step_pins.py``.
"""

from __future__ import annotations

from collections import deque
from fractions import Fraction

import numpy as np

__all__ = ["step_tables", "norm_rope", "verify"]


def step_tables(lens, counts, tables, held, shared, ring, state, K, rows):
    """Returns a dict of the outputs of one step, ``tables`` and ``ring``
    being the updated copies."""
    S, width = tables.shape
    head, tail = int(state[0]), int(state[1])
    R = len(ring)
    lens = [int(x) for x in lens]
    counts = [int(x) for x in counts]
    held = [int(x) for x in held]
    shared = [int(x) for x in shared] if shared is not None else [0] * S
    need = [-(-(L + max(c, 0)) // K) for L, c in zip(lens, counts)]
    invalid = head < 0 or not 0 <= tail - head <= R
    for s in range(S):
        invalid |= (lens[s] < 0 or counts[s] < -1 or not 0 <= held[s] <= width or shared[s] < 0
                    or lens[s] > held[s] * K or need[s] > width)
    total = sum(max(c, 0) for c in counts) if not invalid else 0
    take = sum(max(0, need[s] - held[s]) for s in range(S) if counts[s] >= 0) if not invalid else 0
    give = sum(max(0, held[s] - shared[s]) for s in range(S) if counts[s] < 0) if not invalid else 0
    code = 0
    if invalid or tail + give - head > R:
        code = 3
    elif total > rows:
        code = 2
    elif take > tail - head:
        code = 1
    out = dict(tables=tables.copy(), ring=ring.copy(), positions=np.full(rows, -1, np.int32),
               slots=np.full(rows, -1, np.int64), totals=[code, total, take, give])
    if code:
        return dict(out, context_lens=lens, cu_seqlens=[0] * (S + 1), cu_blocks=[0] * (S + 1),
                    held=held, state=[head, tail])
    free = deque(int(ring[i % R]) for i in range(head, tail))
    ctx, cu, cb, held2 = [], [0], [0], []
    t = 0
    for s in range(S):
        if counts[s] < 0:
            ctx.append(0)
            held2.append(0)
            cu.append(cu[-1])
            cb.append(cb[-1])
            for b in range(shared[s], held[s]):
                out["ring"][tail % R] = tables[s, b]
                tail += 1
            continue
        h = held[s]
        while h < need[s]:
            out["tables"][s, h] = free.popleft()
            head += 1
            h += 1
        for p in range(lens[s], lens[s] + counts[s]):
            out["positions"][t] = p
            out["slots"][t] = int(out["tables"][s, p // K]) * K + p % K
            t += 1
        ctx.append(lens[s] + counts[s])
        cu.append(t)
        cb.append(cb[-1] + h - held[s])
        held2.append(h)
    return dict(out, context_lens=ctx, cu_seqlens=cu, cu_blocks=cb, held=held2,
                state=[head, tail])


def norm_rope(row, weight, eps, position, inv_or_table, interleaved=False):
    """One head row (float64): norm (``weight`` None: none), then rotation by
    the row ``position`` of the table [positions, rot] (cosines, then sines)."""
    y = [float(x) for x in row]
    D = len(y)
    if weight is not None:
        inv = 1.0 / np.sqrt(sum(x * x for x in y) / D + eps)
        y = [x * inv * float(w) for x, w in zip(y, weight)]
    cs = inv_or_table[position]
    half = len(cs) // 2
    out = list(y)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cs[i]), float(cs[half + i])
        out[a] = y[a] * c - y[b] * s
        out[b] = y[b] * c + y[a] * s
    return np.array(out)


def _count(w):
    w = float(w)
    if not w > 0.0:            # negative, zero, NaN
        return 0
    return int(min(w, 1.0) * 2**40)


def verify(target, draft, tokens, uniforms, cu, max_query):
    """``target`` float32 [T, V]; ``draft`` float32 [S, N, V] or None; returns
    (out_tokens [S, max_query], num_new [S])."""
    S, V = len(cu) - 1, target.shape[1]
    out = np.full((S, max_query), -1, np.int64)
    new = np.zeros(S, np.int64)
    for s in range(S):
        c, r = int(cu[s]), int(cu[s + 1] - cu[s])
        if r == 0:
            continue
        a = 0
        while a < r - 1:
            d = int(tokens[c + 1 + a])
            if not 0 <= d < V:
                break
            q = Fraction(float(draft[s, a, d])) if draft is not None else Fraction(1)
            if not Fraction(float(uniforms[c + a])) * q < Fraction(float(target[c + a, d])):
                break
            out[s, a] = d
            a += 1
        p = target[c + a]
        counts = None
        if a < r - 1:
            d = int(tokens[c + 1 + a])
            if 0 <= d < V:
                if draft is not None:
                    counts = [_count(np.float32(x) - np.float32(y)) for x, y in zip(p, draft[s, a])]
                else:
                    counts = [0 if x == d else _count(w) for x, w in enumerate(p)]
        if counts is None or sum(counts) == 0:
            counts = [_count(w) for w in p]
        total = sum(counts)
        if total:
            below = total * int(float(uniforms[c + r - 1]) * 2**24) // 2**24
            run = 0
            for x, w in enumerate(counts):
                run += w
                if run > below:
                    out[s, a] = x
                    break
        new[s] = a + 1
    return out, new
