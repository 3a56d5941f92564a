"""Pins of oracle/step.py against things other than itself: the block manager
and the slot-mapping oracle, closed forms of the rotation, the distribution
that draft verification must preserve, planted mistakes."""

import math

import numpy as np
import pytest

import oracle
from oracle import step as S
from paged_kv_cache_115_gb300.blockmgr import BlockPool, SeqBlocks


def test_tables_match_the_block_manager_and_the_slot_oracle():
    """Several steps of growth against SeqBlocks drawing from the same order
    of free blocks (a queue), and oracle.slot_mapping on the result."""
    rng = np.random.default_rng(0)
    K, R, n = 4, 64, 5
    order = rng.permutation(R).astype(np.int32)
    tables = np.full((n, 12), -9, np.int32)
    lens, held, state, ring = [0] * n, [0] * n, [0, R], order.copy()
    want = [[] for _ in range(n)]
    queue = list(order)
    for _ in range(4):
        counts = [int(x) for x in rng.integers(0, 9, n)]
        o = S.step_tables(lens, counts, tables, held, None, ring, state, K, 64)
        assert o["totals"][0] == 0
        for s in range(n):
            while len(want[s]) * K < lens[s] + counts[s]:
                want[s].append(int(queue.pop(0)))
            assert list(o["tables"][s, :len(want[s])]) == want[s]
            assert o["held"][s] == len(want[s])
        pos = [p for s in range(n) for p in range(lens[s], lens[s] + counts[s])]
        seq = [s for s in range(n) for _ in range(counts[s])]
        T = len(pos)
        assert list(o["positions"][:T]) == pos and (o["positions"][T:] == -1).all()
        if T:
            ref = oracle.slot_mapping(o["tables"][seq], np.array(pos), K)
            assert np.array_equal(o["slots"][:T], ref)
        assert (o["slots"][T:] == -1).all()
        lens, held, state = o["context_lens"], o["held"], o["state"]
        tables, ring = o["tables"], o["ring"]
    sb = SeqBlocks(BlockPool(8, seed=1), K)     # the manager's own count of blocks for a length
    sb.grow_to(9)
    assert len(sb.mapping) == 3 == -(-9 // K)


def test_blocks_of_finished_requests_come_back():
    tables = np.array([[5, 6, 7], [8, 9, -1]], np.int32)
    ring = np.array([1, 2, 0, 0, 0, 0], np.int32)
    o = S.step_tables([10, 5], [-1, 4], tables, [3, 2], [1, 0], ring, [0, 2], 4, 8)
    assert o["totals"] == [0, 4, 1, 2]
    assert list(o["ring"][2:4]) == [6, 7] and o["state"] == [1, 4]     # block 5 is shared
    assert o["held"] == [0, 3] and o["context_lens"] == [0, 9]
    assert list(o["tables"][1]) == [8, 9, 1]
    # given back and taken later, in that order
    o2 = S.step_tables(o["context_lens"], [9, 0], o["tables"], o["held"], None, o["ring"],
                       o["state"], 4, 9)
    assert list(o2["tables"][0]) == [2, 6, 7] and o2["state"] == [4, 4]


@pytest.mark.parametrize("change,code", [
    (dict(state=[0, 1]), 1), (dict(rows=3, state=[0, 2]), 2), (dict(lens=[9, -1]), 3), (dict(counts=[-2, 4]), 3),
    (dict(held=[4, 2]), 3), (dict(lens=[13, 5]), 3), (dict(counts=[4, 9]), 3),
    (dict(state=[3, 2]), 3), (dict(shared=[-1, 0]), 3), (dict(state=[0, 7]), 3)])
def test_refused_steps_change_nothing(change, code):
    a = dict(lens=[9, 5], counts=[-1, 4], held=[3, 2], shared=None, state=[0, 4], rows=8)
    if code == 1:
        a.update(lens=[0, 0], held=[0, 0], counts=[5, 3])
    a.update(change)
    tables = np.arange(6, dtype=np.int32).reshape(2, 3)
    ring = np.arange(6, dtype=np.int32)
    o = S.step_tables(a["lens"], a["counts"], tables, a["held"], a["shared"], ring, a["state"], 4,
                      a["rows"])
    assert o["totals"][0] == code
    assert np.array_equal(o["tables"], tables) and np.array_equal(o["ring"], ring)
    assert o["held"] == a["held"] and o["state"] == a["state"] and o["cu_seqlens"] == [0, 0, 0]


def _table(n, rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(n)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(3)
    D, rot = 16, 12
    t = _table(50, rot)
    x, y = rng.standard_normal(D), rng.standard_normal(D)
    # position 0 is the identity; lengths stay; scores depend on the distance alone
    assert np.allclose(S.norm_rope(x, None, 0, 0, t, interleaved), x)
    a = S.norm_rope(x, None, 0, 7, t, interleaved)
    assert np.isclose((a * a).sum(), (x * x).sum()) and np.array_equal(a[rot:], x[rot:])
    d1 = S.norm_rope(x, None, 0, 30, t, interleaved) @ S.norm_rope(y, None, 0, 25, t, interleaved)
    d2 = S.norm_rope(x, None, 0, 12, t, interleaved) @ S.norm_rope(y, None, 0, 7, t, interleaved)
    assert np.isclose(d1, d2)
    # two turns add up
    b = S.norm_rope(S.norm_rope(x, None, 0, 4, t, interleaved), None, 0, 3, t, interleaved)
    assert np.allclose(a, b)
    # the other pairing is another function
    assert not np.allclose(a, S.norm_rope(x, None, 0, 7, t, not interleaved))


def test_norm_closed_forms():
    t = _table(2, 8)
    x = np.arange(1.0, 9.0)
    y = S.norm_rope(x, np.ones(8), 0.0, 0, t)
    assert np.isclose((y * y).mean(), 1.0)
    assert np.allclose(S.norm_rope(4 * x, np.ones(8), 0.0, 0, t), y)
    assert np.allclose(S.norm_rope(x, np.full(8, 2.0), 0.0, 0, t), 2 * y)
    assert np.array_equal(S.norm_rope(np.zeros(8), np.ones(8), 1e-6, 1, t), np.zeros(8))


def test_verification_keeps_the_targets_distribution():
    """Summed exactly over a grid of random numbers, the first token follows
    the target whatever the draft's distribution: P(token = x) = p(x)."""
    p = np.array([0.5, 0.25, 0.125, 0.125], np.float32)
    q = np.array([0.125, 0.5, 0.25, 0.125], np.float32)
    n = 64
    got = np.zeros(4)
    for d in range(4):                              # the draft proposes d with q(d)
        for i in range(n):
            for j in range(n):
                u = np.array([(i + 0.5) / n, (j + 0.5) / n], np.float32)
                out, new = S.verify(np.stack([p, p]), q[None, None], [0, d], u, [0, 2], 2)
                got[out[0, 0]] += float(q[d]) / n / n
                assert new[0] == (2 if out[0, 0] == d and u[0] * q[d] < p[d] else 1)
    assert np.abs(got - p).max() < 1.0 / n


def test_verification_small_cases():
    p = np.array([[0.0, 1.0, 0.0], [0.25, 0.25, 0.5]], np.float32)
    q = np.array([[[0.5, 0.5, 0.0]]], np.float32)
    half = np.array([0.5, 0.6], np.float32)
    out, new = S.verify(p, q, [0, 1], half, [0, 2], 3)      # accepted: 0.5 * 0.5 < 1
    assert list(out[0]) == [1, 2, -1] and new[0] == 2       # 0.6 falls into [0.5, 1)
    out, new = S.verify(p, q, [0, 0], half, [0, 2], 3)      # refused: p(0) = 0
    assert list(out[0]) == [1, -1, -1] and new[0] == 1
    out, new = S.verify(p, None, [0, 2], half, [0, 2], 3)   # without probabilities: 0.5 < 0 fails
    assert list(out[0]) == [1, -1, -1]
    out, new = S.verify(p, q, [0, 7], half, [0, 2], 3)      # outside the vocabulary
    assert list(out[0]) == [1, -1, -1]
    # p below q everywhere: drawn from p itself
    out, new = S.verify(np.array([[0.25, 0.25, 0.5]] * 2, np.float32),
                        np.array([[[0.5, 0.5, 1.0]]], np.float32), [0, 0],
                        np.array([0.9, 0.3], np.float32), [0, 2], 2)
    assert list(out[0]) == [1, -1]
    out, new = S.verify(p, np.concatenate([q, q]), [0, 1], half, [0, 0, 2], 3)   # a sequence without rows
    assert list(out[0]) == [-1, -1, -1] and new[0] == 0 and new[1] == 2


def test_ties_and_borders_of_the_draw():
    p = np.array([[0.25, 0.25, 0.25, 0.25]], np.float32)
    for x in range(4):
        lo = np.array([x * 0.25], np.float32)                # inclusive lower border
        hi = np.array([np.nextafter(np.float32((x + 1) * 0.25), np.float32(0))], np.float32)
        assert S.verify(p, None, [0], lo, [0, 1], 1)[0][0, 0] == x
        assert S.verify(p, None, [0], hi, [0, 1], 1)[0][0, 0] == x
    z = np.array([[0.0, 0.5, 0.0, 0.5, 0.0]], np.float32)
    assert S.verify(z, None, [0], np.array([0.0], np.float32), [0, 1], 1)[0][0, 0] == 1
    assert math.isclose(S._count(np.float32(1.0)), 2**40) and S._count(np.nan) == 0
    assert S._count(-1.0) == 0 and S._count(7.0) == 2**40
