"""Beam selection and forks of block tables on the GPU against the oracle:
tokens, parents, tables, rings and copies equal; scores within a float32
rounding and the error of the sums."""

import numpy as np
import pytest
import torch

from oracle import beam as OB

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def check_select(ops, logits, scores, N, finished=None, eos=-1, **kw):
    got = ops.beam_select(logits.to(DEV), scores.to(DEV), N,
                          finished=None if finished is None else finished.to(DEV), eos_token=eos, **kw)
    t, p, s, f = (x.cpu().numpy() for x in got)
    wt, wp, ws, wf = OB.beam_select(logits.double().numpy(), scores.double().numpy(), N,
                                    None if finished is None else finished.numpy(), eos)
    assert np.array_equal(p, wp) and np.array_equal(t, wt) and np.array_equal(f, wf)
    none = np.isneginf(ws)
    assert np.array_equal(np.isneginf(s), none)
    # a float32 rounding of the score, and the sum's terms: 2^-22 from the exponential,
    # 2^-24 each from its argument's two roundings (|x - m| log2 e below 64 where a term
    # counts) and up to 2^-24 for each of ~80 additions
    with np.errstate(invalid="ignore"):
        err = np.abs(s.astype(np.float64) - ws)[~none]
    assert (err <= np.abs(ws[~none]) * 2.0 ** -24 + 2.0 ** -22 + 128 * 2.0 ** -24 + 80 * 2.0 ** -24).all()
    return got


def rand(R, B, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn((R * B, V), generator=g) * spread).to(dtype)
    return logits, -4 * torch.rand((R, B), generator=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,B,V,N", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 40, 8), (3, 4, 1000, 4), (1, 8, 4095, 16),
                                     (2, 5, 4097, 32), (1, 32, 16391, 32), (5, 2, 50021, 4), (40, 8, 33000, 8),
                                     (1, 2, 131072, 7)])
def test_select(ops, R, B, V, N, dtype):
    logits, scores = rand(R, B, V, dtype, seed=V + B)
    check_select(ops, logits, scores, N)
    g = torch.Generator().manual_seed(B)
    finished = torch.rand((R, B), generator=g) < 0.4
    check_select(ops, logits, scores, N, finished=finished, eos=V // 2)
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead,pad", [(1, 0), (3, 5), (0, 7)])
def test_select_rows_anywhere(ops, lead, pad, dtype):
    # neighbours of a row hold larger values
    R, B, V = 3, 2, 999
    logits, scores = rand(R, B, V, dtype, seed=lead + 10 * pad)
    wide = torch.full((R * B, lead + V + pad), 50.0, dtype=dtype)
    wide[:, lead:lead + V] = logits
    wide = wide.to(DEV)[:, lead:lead + V]
    a = ops.beam_select(wide, scores.to(DEV), 6)
    b = check_select(ops, logits, scores, 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])
    # (other threads add the terms: the bound of check_select, twice)
    assert (a[2] - b[2]).abs().max() <= 2 * (8 * 2.0 ** -22 + 208 * 2.0 ** -24)


@pytest.mark.parametrize("V", [700, 5000, 40000])
def test_select_ties(ops, V):
    # one value everywhere; then a few above; whole beams alike
    R, B, N = 2, 3, 9
    scores = torch.tensor([[-1.0, -1.0, -2.0], [-3.0, -1.0, -1.0]])
    logits = torch.full((R * B, V), 0.25)
    t, p, _, _ = ops.beam_select(logits.to(DEV), scores.to(DEV), N)
    assert t.cpu().tolist() == [list(range(N))] * 2 and p.cpu().tolist() == [[0] * N, [1] * N]
    logits[:, V - 3] = 1.5
    logits[:, 17] = 1.5
    for dtype in (torch.float32, torch.bfloat16):
        t, p, _, _ = ops.beam_select(logits.to(dtype).to(DEV), scores.to(DEV), N)
        # (rows of 40000 and 5000 values start on 16-byte boundaries, those of 700 do in float32)
        if V % 8 == 0 or dtype == torch.float32:
            assert t.cpu()[0, :4].tolist() == [17, V - 3, 17, V - 3] and p.cpu()[0, :4].tolist() == [0, 0, 1, 1]
            assert t.cpu()[1, :4].tolist() == [17, V - 3, 17, V - 3] and p.cpu()[1, :4].tolist() == [1, 1, 2, 2]
    # both zeros are equal
    z = torch.zeros((1, V))
    z[0, ::2] = -0.0
    t, _, _, _ = ops.beam_select(z.to(DEV), torch.zeros((1, 1), device=DEV), 5)
    assert t.cpu().tolist() == [[0, 1, 2, 3, 4]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_masks(ops, dtype):
    R, B, V, N = 3, 4, 20000, 6
    logits, scores = rand(R, B, V, dtype, seed=1)
    logits[0] = float("-inf")                                   # a beam without candidates
    logits[1, 5:] = float("-inf")                               # a few tokens
    logits[2, :] = float("-inf")
    logits[2, 19999] = torch.finfo(dtype).min                   # one, at the lowest value
    logits[4:8] = float("-inf")                                 # a request without any
    logits[8:12, 100:] = torch.finfo(dtype).min
    scores[2, 1] = float("-inf")
    check_select(ops, logits, scores, N)
    first = torch.full((R, B), float("-inf"))
    first[:, 0] = 0
    check_select(ops, logits, first, N)
    assert ops.get_device_error() == 0


def test_select_first_step_of_one_beam(ops):
    logits, _ = rand(4, 1, 3000, torch.float32, seed=9)
    check_select(ops, logits, torch.zeros((4, 1)), 8)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_select_rows_that_are_not_finite(ops, bad):
    logits, scores = rand(2, 2, 5000, torch.float32, seed=2)
    logits[1, 4321] = bad
    check_select(ops, logits, scores, 4)
    assert ops.get_device_error() == 9
    scores[1, 0] = bad
    logits[1, 4321] = 0
    t, p, s, f = ops.beam_select(logits.to(DEV), scores.to(DEV), 4)
    assert (p[1] == 1).all() and torch.isfinite(s).all()
    assert ops.get_device_error() == 0


def test_select_wide_scores(ops):
    # values of all sizes, the sums far apart
    logits, scores = rand(2, 4, 30000, torch.float32, seed=3, spread=30.0)
    check_select(ops, logits, scores * 1000, 12)


def test_select_outputs_and_runs_alike(ops):
    logits, scores = rand(6, 4, 9000, torch.bfloat16, seed=4)
    logits, scores = logits.to(DEV), scores.to(DEV)
    a = ops.beam_select(logits, scores, 8)
    o = [torch.empty_like(x) for x in a]
    o[3] = torch.empty((6, 8), dtype=torch.uint8, device=DEV)
    ws = torch.full((ops.beam_select_workspace_bytes(6, 4, 9000, 8),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        b = ops.beam_select(logits, scores, 8, tokens=o[0], parents=o[1], scores_out=o[2], finished_out=o[3],
                            workspace=ws)
        assert b[0] is o[0]
        for x, y in zip(a, b):
            assert torch.equal(x, y.to(x.dtype))


# ---------------------------------------------------------------------------

def beam_rows(R, B, K, lo, hi, own, width, rng, dead=0.0):
    """Groups whose rows share whole blocks and part ways, and the free ring."""
    S = R * B
    lens, held = np.zeros(S, np.int32), np.zeros(S, np.int32)
    tables = np.full((S, width), -7, np.int32)
    nb = S * width + 5
    order = list(rng.permutation(nb).astype(np.int32))
    for g in range(R):
        common = int(rng.integers(lo, hi + 1)) // K
        rows = [order.pop() for _ in range(common)]
        for b in range(B):
            s = g * B + b
            if rng.random() < dead:
                continue
            lens[s] = min(common * K + int(rng.integers(0, own + 1)), width * K)
            held[s] = min(width, -(-int(lens[s]) // K) + int(rng.integers(0, 2)))
            lens[s] = min(lens[s], held[s] * K)
            for c in range(held[s]):
                tables[s, c] = rows[c] if c < common else order.pop()
    size = nb + 3
    head = int(rng.integers(0, 4 * size))
    ring = np.full(size, -9, np.int32)
    for i, x in enumerate(order):
        ring[(head + i) % size] = x
    return lens, held, tables, ring, np.array([head, head + len(order)], np.int64), nb


def check_fork(ops, parents, lens, held, shared, tables, ring, state, K, in_place):
    d = [torch.from_numpy(np.array(x)).to(DEV) for x in (parents, lens, held, tables, ring, state)]
    sh = None if shared is None else torch.from_numpy(shared).to(DEV)
    out_tables = None
    if in_place:
        kw = dict(lens_out=d[1], held_out=d[2], ring_state_out=d[5])
    else:
        out_tables = np.full_like(tables, -3)
        kw = dict(block_tables_out=torch.from_numpy(out_tables).to(DEV))
    o = ops.fork_tables(d[0], d[1], d[2], d[3], d[4], d[5], K, shared=sh, **kw)
    w = OB.fork_tables(parents, lens, held, shared, tables, ring, state, K, out_tables)
    assert o["totals"].cpu().tolist() == w["totals"]
    assert np.array_equal(o["block_tables_out"].cpu().numpy(), w["tables"])
    assert o["lens_out"].cpu().tolist() == w["lens"] and o["held_out"].cpu().tolist() == w["held"]
    assert o["ring_state_out"].cpu().tolist() == w["state"]
    assert np.array_equal(d[4].cpu().numpy(), w["ring"])
    assert o["pairs"].cpu().tolist() == [list(map(int, p)) for p in w["pairs"]]
    assert ops.get_device_error() == (7 if w["totals"][0] == 3 else 0)
    return o, w


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("R,B,K,lo,hi,own,width", [(1, 1, 16, 0, 40, 9, 4), (1, 4, 16, 20, 90, 30, 9),
                                                   (7, 5, 8, 0, 100, 60, 24), (3, 8, 1, 5, 60, 8, 80),
                                                   (2, 32, 16, 100, 900, 300, 80), (40, 3, 32, 0, 4000, 500, 150),
                                                   (3, 4, 4, 1000, 2300, 200, 700), (300, 2, 16, 3, 50, 20, 6)])
def test_fork(ops, R, B, K, lo, hi, own, width, in_place):
    rng = np.random.default_rng(R * 1000 + B + K)
    for dead, shared in ((0.0, False), (0.3, True)):
        lens, held, tables, ring, state, _ = beam_rows(R, B, K, lo, min(hi, (width - 1) * K - own), own, width, rng,
                                                       dead)
        parents = rng.integers(-1 if dead else 0, B, (R, B)).astype(np.int32)
        sh = np.repeat(rng.integers(0, 3, R), B).astype(np.int32) if shared else None
        check_fork(ops, parents, lens, held, sh, tables, ring, state, K, in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("what", ["parent", "parent low", "lens", "lens low", "held", "shared", "head", "tail", "few",
                                  "ring"])
def test_fork_refusals(ops, what, in_place):
    rng = np.random.default_rng(11)
    R, B, K, width = 6, 4, 16, 12
    lens, held, tables, ring, state, _ = beam_rows(R, B, K, 30, 100, 40, width, rng)
    lens = np.minimum(lens // K * K + 3, held * K).astype(np.int32)
    parents = np.zeros((R, B), np.int32)
    sh = np.zeros(R * B, np.int32)
    if what == "parent":
        parents[3, 2] = B
    elif what == "parent low":
        parents[3, 2] = -2
    elif what == "lens":
        lens[9] = held[9] * K + 1
    elif what == "lens low":
        lens[9] = -1
    elif what == "held":
        held[9] = width + 1
    elif what == "shared":
        sh[9] = -1
    elif what == "head":
        state[0] = -1
    elif what == "tail":
        state[1] = state[0] - 1
    elif what == "few":
        state[1] = state[0] + 2
    else:
        state[1] = state[0] + len(ring)
    o, w = check_fork(ops, parents, lens, held, sh, tables, ring, state, K, in_place)
    assert w["totals"][0] == (1 if what == "few" else 3)


def test_fork_whole_requests_end(ops):
    rng = np.random.default_rng(12)
    R, B, K, width = 5, 4, 16, 20
    lens, held, tables, ring, state, nb = beam_rows(R, B, K, 60, 200, 60, width, rng)
    parents = np.full((R, B), -1, np.int32)
    o, w = check_fork(ops, parents, lens, held, None, tables, ring, state, K, True)
    distinct = len({int(x) for s in range(R * B) for x in tables[s, :held[s]]})
    assert w["totals"] == [0, 0, 0, distinct]


@pytest.mark.parametrize("fmt", ["bf16", "f32", "fp8", "int8", "k16v8", "int4"])
@pytest.mark.parametrize("layers", [0, 3])
@pytest.mark.parametrize("H,D,K", [(2, 64, 16), (3, 128, 5)])
def test_fork_copy(ops, fmt, layers, H, D, K):
    if layers and fmt in ("fp8", "int8", "k16v8"):
        pytest.skip("one-byte pools: a layer a call")
    g = torch.Generator().manual_seed(H + K)
    nb, S = 9, 5
    lead = (layers,) if layers else ()
    wide = {"bf16": 2 * D, "f32": 4 * D, "k16v8": 2 * D, "int4": D // 2}.get(fmt, D)
    raw_k = torch.randint(0, 256, (*lead, nb, K, H, wide), generator=g, dtype=torch.uint8)
    raw_v = torch.randint(0, 256, (*lead, nb, K, H, D if fmt == "k16v8" else wide), generator=g, dtype=torch.uint8)
    kc, vc = raw_k.to(DEV), raw_v.to(DEV)
    quant, ks, vs = None, None, None
    if fmt == "int4":
        ks, vs = (torch.randint(-32768, 32767, (*lead, nb, H, K, 2), generator=g, dtype=torch.int16) for _ in range(2))
    elif fmt == "int8":
        ks, vs = (torch.randint(-2**31, 2**31 - 1, (nb * K,), generator=g, dtype=torch.int32) for _ in range(2))
    dks, dvs = (None if t is None else t.to(DEV) for t in (ks, vs))
    typed_k, typed_v = kc, vc
    if fmt == "int4":
        quant = ops.kv_quant("int4", k_token_scales=dks.view(torch.bfloat16), v_token_scales=dvs.view(torch.bfloat16))
    elif fmt == "int8":
        quant = ops.kv_quant("int8", k_token_scales=dks.view(torch.float32), v_token_scales=dvs.view(torch.float32))
    elif fmt in ("fp8", "k16v8"):
        quant = ops.kv_quant(fmt)
        typed_k = kc.view(torch.bfloat16) if fmt == "k16v8" else kc
    else:
        typed_k, typed_v = (t.view(torch.bfloat16 if fmt == "bf16" else torch.float32) for t in (kc, vc))
    pairs = torch.tensor([[3, 0], [-1, -1], [8, 7], [2, 5], [6, 1]])
    lens = torch.tensor([K + 1, 7, 2 * K - 1, 3 * K, 4], dtype=torch.int32)     # the fourth: no tokens
    ops.kv_fork_copy(typed_k, typed_v, pairs.to(DEV), lens.to(DEV), quant=quant)
    assert ops.get_device_error() == 0
    for (a, b), n in zip(pairs.tolist(), lens.tolist()):
        if a < 0:
            continue
        n %= K
        for t in (raw_k, raw_v):
            t[..., b, :n, :, :] = t[..., a, :n, :, :]
        for t in (ks, vs):
            if fmt == "int4":
                t[..., b, :, :n, :] = t[..., a, :, :n, :]
            elif fmt == "int8":
                t.view(nb, K)[b, :n] = t.view(nb, K)[a, :n]
    assert torch.equal(kc.cpu(), raw_k) and torch.equal(vc.cpu(), raw_v)
    if ks is not None:
        assert torch.equal(dks.cpu(), ks) and torch.equal(dvs.cpu(), vs)


def test_fork_copy_pairs_out_of_range(ops):
    kc = torch.randn((4, 8, 1, 64), device=DEV)
    vc, want = kc.clone(), kc.clone()
    lens = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    for pair in ([4, 0], [0, 4], [-1, 2], [1, -1], [-2, -2], [2**40, 1]):
        ops.kv_fork_copy(kc, vc, torch.tensor([pair], device=DEV), lens)
        assert ops.get_device_error() == 3
        assert torch.equal(kc, want)
