"""GPU parity of the step tables and of draft verification against
oracle/step.py: whole numbers, equal in every element."""

import numpy as np
import pytest
import torch

from oracle import step as O

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device=DEV)


def tables_problem(rng, S, K, new_hi, over=0.2, shared_hi=2, spare=8, head=0):
    lens = rng.integers(0, 6 * K, S)
    held = -(-lens // K) + rng.integers(0, 3, S)            # some rows hold more than they need
    counts = rng.integers(0, new_hi + 1, S)
    counts[rng.random(S) < over] = -1
    shared = np.minimum(rng.integers(0, shared_hi + 1, S), held)
    width = int(held.max(initial=0)) + -(-new_hi // K) + 8
    blocks = int(S * width + spare)
    order = rng.permutation(blocks)
    tables = np.full((S, width), -77, np.int32)
    at = 0
    for s in range(S):
        tables[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
    ring = np.full(blocks, -5, np.int32)
    free = order[at:]
    for i, b in enumerate(free):
        ring[(head + i) % blocks] = b
    return dict(lens=lens, counts=counts, tables=tables, held=held, shared=shared, ring=ring,
                state=[head, head + len(free)], K=K, blocks=blocks,
                total=int(np.maximum(counts, 0).sum()))


def check_tables(ops, pb, rows, in_place=False, use_shared=True):
    want = O.step_tables(pb["lens"], pb["counts"], pb["tables"], pb["held"],
                         pb["shared"] if use_shared else None, pb["ring"], pb["state"], pb["K"],
                         rows)
    t = dict(lens=dev(pb["lens"]), counts=dev(pb["counts"]), rows=dev(pb["tables"]),
             held=dev(pb["held"]), ring=dev(pb["ring"]), state=dev(pb["state"], torch.int64),
             shared=dev(pb["shared"]) if use_shared else None)
    more = dict(context_lens=t["lens"], held_out=t["held"], ring_state_out=t["state"]) \
        if in_place else {}
    o = ops.step_tables(t["lens"], t["counts"], t["rows"], t["held"], t["ring"], t["state"],
                        pb["K"], pb["blocks"], shared=t["shared"], num_tokens=rows, **more)
    code = ops.get_device_error()
    assert code == (7 if want["totals"][0] >= 2 else 0)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    assert list(got["totals"][:1]) == want["totals"][:1]
    if want["totals"][0] < 3:
        assert list(got["totals"]) == want["totals"]
    assert np.array_equal(t["rows"].cpu().numpy(), want["tables"])
    assert np.array_equal(t["ring"].cpu().numpy(), want["ring"])
    assert np.array_equal(got["positions"], want["positions"])
    assert np.array_equal(got["slots"], want["slots"])
    for a, b in (("context_lens", "context_lens"), ("cu_seqlens", "cu_seqlens"),
                 ("cu_blocks", "cu_blocks"), ("held_out", "held"), ("ring_state_out", "state")):
        assert list(got[a]) == [int(x) for x in want[b]], a
    return want


@pytest.mark.parametrize("S", [1, 2, 31, 33, 1023, 1025, 2500])
@pytest.mark.parametrize("K", [1, 7, 16])
def test_tables(ops, S, K):
    rng = np.random.default_rng(100 * S + K)
    pb = tables_problem(rng, S, K, 5)
    check_tables(ops, pb, pb["total"] + 3)
    check_tables(ops, pb, pb["total"], in_place=True)


@pytest.mark.parametrize("K", [8, 16, 24, 64])
def test_tables_long_prompts(ops, K):
    """More token rows than one CTA does itself; the ring wraps around."""
    rng = np.random.default_rng(K)
    pb = tables_problem(rng, 37, K, 900, head=12345)
    assert pb["total"] > 5000
    check_tables(ops, pb, pb["total"] + 100)
    check_tables(ops, pb, pb["total"] + 100, in_place=True, use_shared=False)


def test_tables_no_requests_no_tokens(ops):
    rng = np.random.default_rng(1)
    pb = tables_problem(rng, 3, 4, 0, over=0.0)
    check_tables(ops, pb, 0)
    check_tables(ops, pb, 9)
    pb = tables_problem(rng, 4, 4, 3, over=1.0)                # every request over
    check_tables(ops, pb, 5)
    z = dict(pb, lens=pb["lens"][:0], counts=pb["counts"][:0], held=pb["held"][:0],
             shared=pb["shared"][:0], tables=pb["tables"][:0])
    check_tables(ops, z, 4)


@pytest.mark.parametrize("rows", [50, 6000])
@pytest.mark.parametrize("change", ["blocks", "tokens", "len", "count", "held", "width", "state",
                                    "ring", "pages"])
def test_tables_refused_steps(ops, rows, change):
    rng = np.random.default_rng(5)
    pb = tables_problem(rng, 9, 4, 5, over=0.3)
    if change == "blocks":
        pb["state"] = [3, 3]                                    # no free block at all
    elif change == "tokens":
        rows = pb["total"] - 1
    elif change == "len":
        pb["lens"][3] = -4
    elif change == "count":
        pb["counts"][2] = -2
    elif change == "held":
        pb["held"][0] = pb["tables"].shape[1] + 1
    elif change == "width":
        pb["counts"][4] = 4 * pb["tables"].shape[1] + 1
    elif change == "state":
        pb["state"] = [5, 4]
    elif change == "ring":
        pb["state"] = [0, pb["blocks"]]                         # no room for what comes back
        pb["counts"][:] = -1
        pb["held"][:] = np.maximum(pb["held"], 1)
        pb["shared"][:] = 0
    else:
        pb["lens"][1] = 4 * int(pb["held"][1]) + 1              # cached tokens without a block
    want = check_tables(ops, pb, rows)
    assert want["totals"][0] != 0


def test_tables_bad_free_block(ops):
    """A free block outside the pool: listed, its tokens get slot -1."""
    rng = np.random.default_rng(2)
    pb = tables_problem(rng, 4, 4, 9, over=0.0)
    pb["lens"][:] = 0
    pb["held"][:] = 0
    pb["counts"][:] = [5, 4, 8, 1]
    pb["ring"][2] = pb["blocks"]
    o = ops.step_tables(dev(pb["lens"]), dev(pb["counts"]), dev(pb["tables"]), dev(pb["held"]),
                        dev(pb["ring"]), dev([0, 40], torch.int64), 4, pb["blocks"], num_tokens=18)
    assert ops.get_device_error() == 1
    slots = o["slots"].cpu().numpy()
    assert (slots[5:9] == -1).all() and (np.delete(slots, range(5, 9)) >= 0).all()


def test_tables_in_a_captured_loop(ops):
    """One captured step, replayed: the state lives on the device."""
    rng = np.random.default_rng(8)
    pb = tables_problem(rng, 20, 4, 0, over=0.0, spare=400)
    w = dict(pb)
    t = dict(lens=dev(pb["lens"]), counts=dev(pb["counts"]), rows=dev(pb["tables"]),
             held=dev(pb["held"]), ring=dev(pb["ring"]), state=dev(pb["state"], torch.int64))
    outs = ops.step_tables(t["lens"], t["counts"], t["rows"], t["held"], t["ring"], t["state"], 4,
                           pb["blocks"], num_tokens=64)
    outs.update(context_lens=t["lens"], held_out=t["held"], ring_state_out=t["state"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.step_tables(t["lens"], t["counts"], t["rows"], t["held"], t["ring"], t["state"], 4,
                        pb["blocks"], **outs)
    for _ in range(4):
        counts = rng.integers(0, 4, 20)
        counts[rng.integers(0, 20)] = -1
        t["counts"].copy_(dev(counts))
        graph.replay()
        torch.cuda.synchronize()
        o = O.step_tables(w["lens"], counts, w["tables"], w["held"], None, w["ring"], w["state"],
                          4, 64)
        assert o["totals"][0] == 0
        assert np.array_equal(t["rows"].cpu().numpy(), o["tables"])
        assert np.array_equal(t["ring"].cpu().numpy(), o["ring"])
        assert np.array_equal(outs["slots"].cpu().numpy(), o["slots"])
        assert list(t["lens"].cpu().numpy()) == o["context_lens"]
        assert list(t["state"].cpu().numpy()) == o["state"]
        w = dict(w, lens=o["context_lens"], tables=o["tables"], held=o["held"], ring=o["ring"],
                 state=o["state"])
    assert ops.get_device_error() == 0


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------

def verify_problem(rng, rows, V, dtype=torch.float32, peaked=3.0):
    """Sequences of rows[s] rows (drafts + 1, 0: none)."""
    S, N = len(rows), max(rows) - 1
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    T = int(cu[-1])
    logit = rng.standard_normal((T, V)) * peaked
    p = np.exp(logit - logit.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    q = np.zeros((S, max(N, 1), V))
    tokens = np.full(T, 10**9, np.int64)
    for s in range(S):
        for i in range(rows[s] - 1):
            lg = logit[cu[s] + i] + 0.7 * rng.standard_normal(V)
            e = np.exp(lg - lg.max())
            q[s, i] = e / e.sum()
            tokens[cu[s] + 1 + i] = rng.choice(V, p=q[s, i])
    u = rng.random(T).astype(np.float32)
    u = np.minimum(u, np.float32(0.99999994))
    target = torch.from_numpy(p).to(dtype)
    draft = torch.from_numpy(q).to(dtype)
    return dict(target=target, draft=draft, tokens=tokens, u=u, cu=cu, N=N)


def check_verify(ops, pb, use_draft=True, error=0, target=None, draft=None):
    draft_h = pb["draft"].float().numpy() if use_draft else None
    want, new = O.verify(pb["target"].float().numpy(), draft_h, pb["tokens"], pb["u"], pb["cu"],
                         pb["N"] + 1)
    target = pb["target"].to(DEV) if target is None else target
    if use_draft:
        draft = pb["draft"].to(DEV) if draft is None else draft
    o, n = ops.verify_draft_tokens(target, draft if use_draft else None, dev(pb["tokens"]),
                                   torch.from_numpy(pb["u"]).to(DEV), dev(pb["cu"]), pb["N"] + 1)
    assert ops.get_device_error() == error
    assert np.array_equal(o.cpu().numpy(), want), (o.cpu().numpy() - want).nonzero()
    assert np.array_equal(n.cpu().numpy(), new)
    return want, new


@pytest.mark.parametrize("V", [1, 2, 31, 129, 1000, 4096, 32000, 50021])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify(ops, V, dtype):
    rng = np.random.default_rng(V)
    pb = verify_problem(rng, [5, 1, 0, 3, 2, 5, 4, 1, 5], V, dtype)
    pb["tokens"][pb["tokens"] == 10**9] = 0
    want, new = check_verify(ops, pb)
    if V >= 129:
        assert len(set(new.tolist())) > 2         # refused and accepted ones both occur
    check_verify(ops, pb, use_draft=False)


@pytest.mark.parametrize("rows", [[1], [2], [40, 34, 70]])
def test_verify_few_and_many_drafts(ops, rows):
    """One sequence; more drafts than a warp has lanes, the first refusal late."""
    rng = np.random.default_rng(sum(rows))
    pb = verify_problem(rng, rows, 515)
    pb["tokens"][pb["tokens"] == 10**9] = 0
    check_verify(ops, pb)
    pb["u"][:-1] *= 0.02
    check_verify(ops, pb)


def test_verify_strided_rows(ops):
    """Probabilities cut out of wider tensors, drafts stacked step by step;
    rows that start off a 16-byte boundary."""
    rng = np.random.default_rng(4)
    pb = verify_problem(rng, [4, 3, 4, 1], 2051)
    pb["tokens"][pb["tokens"] == 10**9] = 0
    T = pb["target"].shape[0]
    for pad in (1, 2, 5, 13):
        wide = torch.full((T, 2051 + pad), float("nan"), device=DEV)
        wide[:, pad:] = pb["target"].to(DEV)
        steps = torch.full((3, 4, 2051 + pad), float("nan"), device=DEV)
        steps[:, :, pad:] = pb["draft"].to(DEV).transpose(0, 1)
        check_verify(ops, pb, target=wide[:, pad:], draft=steps.transpose(0, 1)[:, :, pad:])


def test_verify_odd_values(ops):
    """Negative values, NaN, infinities, a draft above the target everywhere,
    rows without weight, random numbers of 0."""
    rng = np.random.default_rng(6)
    pb = verify_problem(rng, [3, 3, 3, 2, 1], 700)
    pb["tokens"][pb["tokens"] == 10**9] = 0
    pb["target"][0, 5] = float("nan")
    pb["target"][1, 7] = -1.0
    pb["target"][2, 9] = float("inf")
    pb["draft"][1] = pb["target"][3:5] * 2
    pb["u"][3] = 0.9999
    pb["u"][5] = 0.0
    pb["u"][10] = 0.0
    check_verify(ops, pb)
    pb["target"][-1] = 0.0
    check_verify(ops, pb, error=8)
    pb["target"][-1, 699] = 1e-30                   # below one unit of the count: no weight either
    check_verify(ops, pb, error=8)
    pb["target"][-1, 699] = 1.0
    pb["tokens"][1] = 700
    check_verify(ops, pb, error=8)
    pb["tokens"][1] = -1
    check_verify(ops, pb, use_draft=False, error=8)


def test_verify_inconsistent_lengths(ops):
    rng = np.random.default_rng(7)
    pb = verify_problem(rng, [3, 2, 4], 64)
    pb["tokens"][pb["tokens"] == 10**9] = 0
    want, new = O.verify(pb["target"].numpy(), pb["draft"].numpy(), pb["tokens"], pb["u"],
                         pb["cu"], 4)
    for s, cu in ((2, [0, 3, 5, 10]), (1, [0, 3, 2, 6]), (2, [0, 3, 5, 4])):
        o, n = ops.verify_draft_tokens(pb["target"].to(DEV), pb["draft"].to(DEV),
                                       dev(pb["tokens"]), torch.from_numpy(pb["u"]).to(DEV),
                                       dev(cu), 4)
        assert ops.get_device_error() == 8
        assert (o[s] == -1).all() and n[s] == 0
        assert np.array_equal(o[0].cpu().numpy(), want[0])


def test_verify_any_cluster_gives_the_same(ops):
    """The same sequence alone (many CTAs) and among hundreds (one CTA each)."""
    rng = np.random.default_rng(9)
    one = verify_problem(rng, [4], 40009)
    one["tokens"][0] = 0
    want, new = check_verify(ops, one)
    S = 400
    pb = dict(target=one["target"].repeat(S, 1), draft=one["draft"].repeat(S, 1, 1),
              tokens=np.tile(one["tokens"], S), u=np.tile(one["u"], S),
              cu=np.arange(S + 1) * 4)
    o, n = ops.verify_draft_tokens(pb["target"].to(DEV), pb["draft"].to(DEV), dev(pb["tokens"]),
                                   torch.from_numpy(pb["u"]).to(DEV), dev(pb["cu"]), 4)
    assert (o.cpu().numpy() == want).all() and (n.cpu().numpy() == new).all()


def test_refused_arguments(ops):
    f = torch.rand((4, 64), device=DEV)
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    cu = dev([0, 2, 4])
    with pytest.raises(ValueError):
        ops.verify_draft_tokens(f, None, i.cpu(), f[:, 0].contiguous(), cu, 2)
    with pytest.raises(TypeError):
        ops.verify_draft_tokens(f, None, i.long(), f[:, 0].contiguous(), cu, 2)
    with pytest.raises(TypeError):
        ops.verify_draft_tokens(f.half(), None, i, f[:, 0].contiguous(), cu, 2)
    with pytest.raises(ValueError):
        ops.verify_draft_tokens(f.t().contiguous().t(), None, i, f[:, 0].contiguous(), cu, 2)
    with pytest.raises(ValueError):
        ops.verify_draft_tokens(f, f.view(2, 2, 64)[:, :1], i, f[:, 0].contiguous(), cu, 3)
    with pytest.raises(ValueError):
        ops.step_tables(i, i, i.view(2, 2), i, i, cu, 4, 4, num_tokens=4)
    with pytest.raises(ValueError):
        ops.step_tables(i, i, i.view(4, 1), i, i, cu[:2].long(), 4, 4)
