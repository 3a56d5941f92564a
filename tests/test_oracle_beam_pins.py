"""Pins of ``oracle/beam.py`` and of the 4-bit format in ``oracle/quant.py``:
hand-made cases, closed forms, brute force."""

import itertools
import math

import numpy as np
import pytest

from oracle import beam as OB
from oracle import quant as Q


def f32_of(bits):
    return (np.asarray(bits, np.uint32) << np.uint32(16)).view(np.float32)


def test_int4_hand_made_rows():
    # 0, 1, .. 15: offset 0, scale 1, codes as they are
    c, s, z = Q.int4_quantize(np.arange(16, dtype=np.float32))
    assert c.tolist() == list(range(16)) and f32_of([s, z]).tolist() == [1, 0]
    # one value: the offset is the value rounded down, a step that reaches back up to it
    c, s, z = Q.int4_quantize(np.full(8, -1.001, np.float32))
    assert f32_of([z])[0] == np.float32(-1.0078125) and (c == 15).all()
    c, s, z = Q.int4_quantize(np.full(8, 2.5, np.float32))
    assert f32_of([s, z]).tolist() == [0, 2.5] and not c.any()
    # halves go to the even code
    c, s, z = Q.int4_quantize(np.array([0, 0.5, 1.5, 2.5, 15], np.float32))
    assert c.tolist() == [0, 0, 2, 2, 15]
    assert Q.int4_pack(np.array([1, 2, 3, 15], np.uint8)).tolist() == [0x21, 0xF3]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_int4_rows_that_are_not_finite(bad):
    c, s, z = Q.int4_quantize(np.array([1, bad, 2, 3], np.float32))
    assert not c.any() and np.isnan(f32_of([s, z])).all()


@pytest.mark.parametrize("seed", range(8))
def test_int4_error_bound(seed):
    # half a step; a scale rounded by 2^-9 moves the 15th code by 15 / 512 of a
    # step more and float32 roundings by far less; an offset stored below the
    # least value keeps every code at 0 or above
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((50, 128)) * 10.0 ** rng.integers(-4, 4, (50, 1))
         + rng.standard_normal((50, 1)) * 10.0 ** rng.integers(-4, 4, (50, 1))).astype(np.float32)
    codes, scales, offsets = Q.int4_quantize(x)
    for row, c, s, z in zip(x, codes, scales, offsets):
        s, z = (float(v) for v in f32_of([s, z]))
        assert z <= row.min() and z >= row.min() - abs(float(row.min())) * 2.0 ** -7
        assert np.abs(z + s * c - row).max() <= (0.5 + 15 / 256) * s + 1e-6 * abs(z)


def test_int4_rows_one_by_one():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((7, 3, 32)) * 10.0 ** rng.integers(-3, 3, (7, 3, 1))).astype(np.float32)
    x[2, 1, 5] = np.nan
    c, s, z = Q.int4_quantize(x)
    for i, j in itertools.product(range(7), range(3)):
        one = Q.int4_quantize(x[i, j])
        assert np.array_equal(one[0], c[i, j]) and one[1] == s[i, j] and one[2] == z[i, j]


def test_int4_write_and_read_back():
    rng = np.random.default_rng(1)
    nb, K, H, D = 5, 4, 2, 8
    kp, vp = (rng.integers(0, 256, (nb, K, H, D // 2)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.integers(0, 65536, (nb, H, K, 2)).astype(np.uint16) for _ in range(2))
    k, v = (rng.standard_normal((3, H, D)).astype(np.float32) for _ in range(2))
    slots = [7, -1, 18]
    out = Q.kv_write_int4(kp, vp, ks, vs, k, v, slots)
    touched = {(1, 3), (4, 2)}
    for b, t, h in itertools.product(range(nb), range(K), range(H)):
        same = (out[0][b, t, h] == kp[b, t, h]).all() and (out[2][b, h, t] == ks[b, h, t]).all()
        if (b, t) not in touched:
            assert same
    for i, s in ((0, 7), (2, 18)):
        for h in range(H):
            c, sc, z = Q.int4_quantize(k[i, h])
            want = float(f32_of([z])[0]) + float(f32_of([sc])[0]) * c
            assert np.array_equal(Q.int4_decode(out[0], out[2], [s], h)[0], want)


def test_int4_attention_is_the_plain_one_on_the_values():
    import oracle
    rng = np.random.default_rng(2)
    nb, K, H, D, S = 6, 4, 2, 32, 2
    pools = [np.zeros((nb, K, H, D // 2), np.uint8) for _ in range(2)]
    scales = [np.zeros((nb, H, K, 2), np.uint16) for _ in range(2)]
    rows = [rng.standard_normal((nb * K, H, D)).astype(np.float32) for _ in range(2)]
    kp, vp, ks, vs = Q.kv_write_int4(*pools, *scales, *rows, range(nb * K))
    q = rng.standard_normal((S, 4, D)).astype(np.float32)
    bt, lens = np.array([[3, 0, 5], [1, 4, 2]], np.int32), [9, 5]
    got = Q.paged_attention_decode_int4(q, kp, vp, ks, vs, bt, lens, 0.3, "f32")
    dense = [np.stack([Q.int4_decode(p, w, range(nb * K), h) for h in range(H)], 1)
             .astype(np.float32).reshape(nb, K, H, D) for p, w in ((kp, ks), (vp, vs))]
    want = oracle.paged_attention_decode(q, *dense, bt, lens, 0.3, "f32")
    assert np.abs(got - want).max() < 1e-6          # (the values rounded to float32)


# ---------------------------------------------------------------------------

def test_select_by_hand():
    # two beams, three tokens; probabilities 1/2, 1/4, 1/4 and 1/8, 1/8, 3/4
    logits = np.log(np.array([[2, 1, 1], [1, 1, 6]], np.float64))
    scores = np.log(np.array([[0.5, 0.25]]))
    t, p, s, f = OB.beam_select(logits, scores, 4, eos=2)
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 2, 1, 2]]
    assert np.allclose(np.exp(s), [[1 / 4, 3 / 16, 1 / 8, 1 / 8]])
    assert f.tolist() == [[False, True, False, True]]


def test_select_finished_masked_and_missing():
    logits = np.array([[0.0, 0.0, -np.inf], [5.0, 1.0, 2.0], [-np.inf] * 3])
    scores = np.array([[-1.0, -0.5, -0.1]])
    t, p, s, f = OB.beam_select(logits, scores, 4, finished=np.array([[False, True, False]]), eos=1)
    assert p.tolist() == [[1, 0, 0, -1]] and t.tolist() == [[1, 0, 1, -1]]
    assert s[0, 0] == -0.5 and s[0, 3] == -np.inf
    assert f.tolist() == [[True, False, True, True]]


@pytest.mark.parametrize("seed", range(5))
def test_select_brute_force(seed):
    rng = np.random.default_rng(seed)
    R, B, V, N = 3, 3, 7, 5
    logits = rng.integers(-2, 3, (R * B, V)).astype(np.float64)      # many ties within a row
    scores = rng.standard_normal((R, B))
    t, p, s, _ = OB.beam_select(logits, scores, N)
    for r in range(R):
        prob = {}
        for b in range(B):
            e = [math.exp(x) for x in logits[r * B + b]]
            for v in range(V):
                prob[(b, v)] = scores[r, b] + math.log(e[v] / sum(e))
        for n in range(N):
            mine = (p[r, n], t[r, n])
            assert abs(prob[mine] - s[r, n]) < 1e-12
            ahead = [k for k in prob if prob[k] > prob[mine] + 1e-12
                     or (abs(prob[k] - prob[mine]) <= 1e-12 and k < mine)]
            assert len(ahead) == n


def test_select_keeps_the_sum_of_probabilities():
    # all candidates of a beam at score 0 add up to 1
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((1, 20))
    _, _, s, _ = OB.beam_select(logits, np.zeros((1, 1)), 20)
    assert abs(np.exp(s).sum() - 1) < 1e-12


# ---------------------------------------------------------------------------

def test_fork_by_hand():
    # K = 4, one group of 3 rows: row 0 of 6 tokens in blocks 10, 11; row 1 of 6 in
    # 10, 12; row 2 of 6 in 10, 13.  Rows 0 and 2 continue row 1, row 1 continues
    # row 2: row 0's block 11 is free, row 2 gets block 20 and a copy of 12.
    tables = np.array([[10, 11, -7], [10, 12, -7], [10, 13, -7]], np.int32)
    o = OB.fork_tables(np.array([[1, 2, 1]]), [6, 6, 6], [2, 2, 2], None, tables,
                       np.array([20, 21, -1, -1], np.int32), [0, 2], 4)
    assert o["tables"].tolist() == [[10, 12, -7], [10, 13, -7], [10, 20, -7]]
    assert o["pairs"] == [[-1, -1], [-1, -1], [12, 20]]
    assert o["state"] == [1, 3] and o["ring"].tolist() == [20, 21, 11, -1]
    assert o["totals"] == [0, 3, 1, 1] and o["held"] == [2, 2, 2]
    # the request ends: every block once, but the shared one
    e = OB.fork_tables(np.array([[-1, -1, -1]]), o["lens"], o["held"], [1, 1, 1], o["tables"],
                       np.array([20, 21, 11, -1, -1, -1, -1, -1], np.int32), o["state"], 4)
    assert e["ring"].tolist()[3:6] == [12, 13, 20] and e["state"] == [1, 6]
    assert e["held"] == [0, 0, 0] and e["totals"] == [0, 0, 0, 3]


def test_fork_full_blocks_need_no_copy():
    tables = np.array([[3, 4, 9], [5, 0, 0]], np.int32)       # row 0: 8 tokens and a spare block
    o = OB.fork_tables(np.array([[0, 0]]), [8, 1], [3, 1], None, tables,
                       np.array([7, 8, 0, 0], np.int32), [0, 2], 4)
    assert o["tables"].tolist() == [[3, 4, 9], [3, 4, 0]] and o["held"] == [3, 2]
    assert o["totals"] == [0, 2, 0, 1] and o["ring"][2] == 5
    assert o["pairs"] == [[-1, -1], [-1, -1]]


@pytest.mark.parametrize("kw,code", [
    (dict(parents=[[0, 2]]), 3), (dict(parents=[[-2, 0]]), 3), (dict(lens=[9, 4]), 3),
    (dict(lens=[-1, 4]), 3), (dict(held=[4, 1]), 3), (dict(shared=[-1, 0]), 3),
    (dict(state=[2, 1]), 3), (dict(state=[0, 5]), 3), (dict(state=[1, 1]), 1),
    (dict(state=[0, 4]), 3), (dict(), 0)])
def test_fork_refusals(kw, code):
    a = dict(parents=[[0, 0]], lens=[6, 4], held=[2, 1], shared=[0, 0],
             tables=np.array([[1, 2, 0], [3, 0, 0]], np.int32), ring=np.array([5, 6, 7, 8], np.int32),
             state=[0, 2], K=4)
    a.update(kw)
    a["parents"] = np.array(a["parents"])
    o = OB.fork_tables(**a)
    assert o["totals"][0] == code
    if code:
        assert np.array_equal(o["tables"], a["tables"]) and o["pairs"] == [[-1, -1]] * 2
        assert o["state"] == list(a["state"]) and np.array_equal(o["ring"], a["ring"])


@pytest.mark.parametrize("seed", range(6))
def test_fork_loses_and_doubles_no_block(seed):
    # many steps of growth and forks: every block is free once or listed, and rows
    # of a group hold the same history as a simulation with copied lists of tokens
    rng = np.random.default_rng(seed)
    R, B, K, width, nb = 2, 3, 4, 12, 80
    tables = np.full((R * B, width), -1, np.int32)
    ring = np.arange(nb, dtype=np.int32)
    state, lens, held = [0, nb], [0] * (R * B), [0] * (R * B)
    text = [[] for _ in range(R * B)]
    content = {}
    for step in range(30):
        parents = rng.integers(0, B, (R, B))
        o = OB.fork_tables(parents, lens, held, None, tables, ring, state, K)
        assert o["totals"][0] == 0
        tables, ring, state, lens, held = (o[k] for k in ("tables", "ring", "state", "lens", "held"))
        for s, (a, b) in enumerate(o["pairs"]):
            if a >= 0:
                for t in range(lens[s] % K):
                    content[(b, t)] = content[(a, t)]
        text = [list(text[g * B + p]) for g in range(R) for p in parents[g]]
        for s in range(R * B):                       # one new token a row
            if lens[s] == held[s] * K:
                tables[s, held[s]] = ring[state[0] % nb]
                state = [state[0] + 1, state[1]]
                held[s] += 1
            content[(int(tables[s, lens[s] // K]), lens[s] % K)] = (step, s)
            text[s].append((step, s))
            lens[s] += 1
            assert [content[(int(tables[s, t // K]), t % K)] for t in range(lens[s])] == text[s]
        free = [int(ring[i % nb]) for i in range(state[0], state[1])]
        listed = {int(x) for s in range(R * B) for x in tables[s, :held[s]]}
        assert sorted(free + list(listed)) == list(range(nb))
