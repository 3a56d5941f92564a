"""Beam search over 4-bit pages as an engine runs it: write, attention with shared
prefixes, selection, fork, copy, step tables, eager and captured, without a host
read in between; and the calls at their edges (streams, two at once, offsets past
32 bits)."""

import numpy as np
import pytest
import torch

from oracle import beam as OB
from oracle import quant as Q
from tests._helpers import as_f64, check_attention, storage

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


class Engine:
    """R requests of B beams, one layer; the model's output is drawn in advance."""

    def __init__(self, ops, R, B, K, H_q, H_kv, D, V, steps, seed):
        g = torch.Generator().manual_seed(seed)
        self.ops, self.R, self.B, self.K, self.V = ops, R, B, K, V
        S = R * B
        self.S, self.D, self.H_q, self.H_kv = S, D, H_q, H_kv
        width, nb = 8, S * 8 + 3
        self.width, self.nb = width, nb
        i32 = torch.int32
        self.kc, self.vc = (torch.zeros((nb, K, H_kv, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
        self.ks, self.vs = (torch.full((nb, H_kv, K, 2), float("nan"), dtype=torch.bfloat16, device=DEV)
                            for _ in range(2))
        self.quant = ops.kv_quant("int4", k_token_scales=self.ks, v_token_scales=self.vs)
        self.lens = torch.zeros(S, dtype=i32, device=DEV)
        self.held = torch.zeros(S, dtype=i32, device=DEV)
        self.tables = torch.full((S, width), -7, dtype=i32, device=DEV)
        self.ring = torch.randperm(nb, generator=g).to(i32).to(DEV)
        self.state = torch.tensor([0, nb], dtype=torch.int64, device=DEV)
        self.one = torch.ones(S, dtype=i32, device=DEV)
        self.scores = torch.full((R, B), float("-inf"), device=DEV)
        self.scores[:, 0] = 0
        self.over = torch.zeros((R, B), dtype=torch.bool, device=DEV)
        self.draws = [dict(q=torch.randn((S, H_q, D), generator=g).to(torch.bfloat16),
                           kv=torch.randn((S, 2 * H_kv * D), generator=g).to(torch.bfloat16),
                           logits=(torch.randn((S, V), generator=g) * 2).to(torch.bfloat16)) for _ in range(steps)]
        self.inp = {k: v.to(DEV) for k, v in self.draws[0].items()}
        self.parents = torch.empty((R, B), dtype=i32, device=DEV)
        self.tokens = torch.empty((R, B), dtype=i32, device=DEV)
        self.scores2, self.over2 = torch.empty_like(self.scores), torch.empty_like(self.over)
        self.out = torch.empty((S, H_q, D), dtype=torch.bfloat16, device=DEV)
        self.pos = torch.empty(S, dtype=i32, device=DEV)
        self.slots = torch.empty(S, dtype=torch.int64, device=DEV)
        self.cu = torch.empty(S + 1, dtype=i32, device=DEV)
        self.cb = torch.empty(S + 1, dtype=i32, device=DEV)
        self.pairs = torch.empty((S, 2), dtype=torch.int64, device=DEV)
        self.tot = torch.empty(4, dtype=i32, device=DEV)
        self.tot2 = torch.empty(4, dtype=i32, device=DEV)
        most = width * K
        self.most = most
        self.ws = torch.empty(ops.attention_quant_workspace_bytes(S, H_q, H_kv, D, K, most, torch.bfloat16, self.quant,
                                                                  share_prefix=True), dtype=torch.uint8, device=DEV)
        self.ws_b = torch.empty(ops.beam_select_workspace_bytes(R, B, V, B), dtype=torch.uint8, device=DEV)
        self.ws_f = torch.empty(ops.fork_workspace_bytes(R, B, width), dtype=torch.uint8, device=DEV)

    def step(self):
        o, J, D = self.ops, self.H_kv, self.D
        o.step_tables(self.lens, self.one, self.tables, self.held, self.ring, self.state, self.K, self.nb,
                      context_lens=self.lens, cu_seqlens=self.cu, cu_blocks=self.cb, positions=self.pos,
                      slots=self.slots, held_out=self.held, ring_state_out=self.state, totals=self.tot)
        kv = self.inp["kv"]
        o.paged_kv_write_quant(kv[:, :J * D].view(self.S, J, D), kv[:, J * D:].view(self.S, J, D), self.slots,
                               self.kc, self.vc, self.quant)
        o.paged_attention_decode_quant(self.inp["q"], self.kc, self.vc, self.tables, self.lens, D ** -0.5, self.quant,
                                       out=self.out, max_context_len=self.most, workspace=self.ws, share_prefix=True)
        o.beam_select(self.inp["logits"], self.scores, self.B, finished=self.over, eos_token=3, tokens=self.tokens,
                      parents=self.parents, scores_out=self.scores2, finished_out=self.over2, workspace=self.ws_b)
        o.fork_tables(self.parents, self.lens, self.held, self.tables, self.ring, self.state, self.K,
                      lens_out=self.lens, held_out=self.held, ring_state_out=self.state, pairs=self.pairs,
                      totals=self.tot2, workspace=self.ws_f)
        o.kv_fork_copy(self.kc, self.vc, self.pairs, self.lens, quant=self.quant)
        self.scores.copy_(self.scores2)
        self.over.copy_(self.over2)


def simulate(e):
    """The same steps with the oracles, from histories copied beam by beam."""
    S, J, D, K = e.S, e.H_kv, e.D, e.K
    text = [([], []) for _ in range(S)]                       # K rows and V rows of each beam
    scores = np.full((e.R, e.B), -np.inf)
    scores[:, 0] = 0
    over = np.zeros((e.R, e.B), bool)
    for d in e.draws:
        kv = d["kv"].float().numpy()
        for s in range(S):
            text[s][0].append(kv[s, :J * D].reshape(J, D))
            text[s][1].append(kv[s, J * D:].reshape(J, D))
        n = [len(t[0]) for t in text]
        nb = sum(-(-x // K) for x in n) + 1
        pool = [np.zeros((nb, K, J, D // 2), np.uint8) for _ in range(2)]
        words = [np.zeros((nb, J, K, 2), np.uint16) for _ in range(2)]
        bt = np.zeros((S, -(-max(n) // K)), np.int32)
        at, rows, slots = 0, ([], []), []
        for s in range(S):
            for c in range(-(-n[s] // K)):
                bt[s, c] = at
                at += 1
            slots += [int(bt[s, t // K]) * K + t % K for t in range(n[s])]
            rows[0].extend(text[s][0]), rows[1].extend(text[s][1])
        kp, vp, ks, vs = Q.kv_write_int4(*pool, *words, np.array(rows[0]), np.array(rows[1]), slots)
        out = Q.paged_attention_decode_int4(storage(d["q"]), kp, vp, ks, vs, bt, n, D ** -0.5, "bf16")
        t, p, sc, ov = OB.beam_select(d["logits"].double().numpy(), scores, e.B, over, 3)
        yield out, t, p, sc
        text = [([], []) if p[s // e.B, s % e.B] < 0 else
                tuple(list(x) for x in text[s // e.B * e.B + p[s // e.B, s % e.B]]) for s in range(S)]
        scores, over = np.where(np.isneginf(sc), -np.inf, sc.astype(np.float32)).astype(np.float64), ov


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("R,B,K,H_q,H_kv,V", [(3, 4, 4, 8, 4, 1000), (2, 3, 8, 7, 1, 257), (1, 8, 16, 16, 2, 4000)])
def test_beam_search(ops, R, B, K, H_q, H_kv, V, captured):
    steps = 20
    e = Engine(ops, R, B, K, H_q, H_kv, 128, V, steps, seed=R + V)
    graph = None
    if captured:
        keep = {k: v.clone() for k, v in vars(e).items() if isinstance(v, torch.Tensor)}
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            e.step()                                          # (loads every kernel)
        side.synchronize()
        for k, v in keep.items():
            getattr(e, k).copy_(v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            e.step()
        for k, v in keep.items():
            getattr(e, k).copy_(v)
    for i, (out, t, p, sc) in enumerate(simulate(e)):
        for k, v in e.draws[i].items():
            e.inp[k].copy_(v)
        graph.replay() if graph else e.step()
        assert e.tot.tolist()[0] == 0 and e.tot2.tolist()[0] == 0
        live = p >= 0
        check_attention(as_f64(e.out), out, "bf16", f"step {i}")
        assert np.array_equal(e.parents.cpu().numpy(), p) and np.array_equal(e.tokens.cpu().numpy(), t)
        assert np.allclose(e.scores.cpu().numpy()[live], sc[live], rtol=0, atol=1e-4)
        # every block is free once or listed
        h, tb = e.held.tolist(), e.tables.cpu().numpy()
        s0, s1 = e.state.tolist()
        ring = e.ring.cpu().numpy()
        free = [int(ring[j % len(ring)]) for j in range(s0, s1)]
        listed = {int(x) for s in range(e.S) for x in tb[s, :h[s]]}
        assert sorted(free + list(listed)) == list(range(e.nb))
    assert ops.get_device_error() == 0


def test_two_streams_at_once(ops):
    # the same calls from two streams, each with buffers and workspaces of its own
    es = [Engine(ops, 2, 4, 8, 8, 8, 128, 3000, 6, seed=s) for s in (5, 6)]
    streams = [torch.cuda.Stream() for _ in es]
    torch.cuda.synchronize()
    want = [[(p, t) for _, t, p, _ in simulate(e)] for e in es]
    got = [[], []]
    for i in range(6):
        for n, (e, s) in enumerate(zip(es, streams)):
            with torch.cuda.stream(s):
                for k, v in e.draws[i].items():
                    e.inp[k].copy_(v)
                e.step()
                got[n].append((e.parents.clone(), e.tokens.clone()))
    torch.cuda.synchronize()
    for n in range(2):
        for (p, t), (wp, wt) in zip(got[n], want[n]):
            assert np.array_equal(p.cpu().numpy(), wp) and np.array_equal(t.cpu().numpy(), wt)


def test_offsets_past_32_bits(ops):
    # a pool of more than 2^32 bytes of codes: the last blocks, written, read and copied
    H, D, K = 16, 128, 16
    nb = (2**32) // (K * H * D // 2) + 64
    kc, vc = (torch.empty((nb, K, H, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((nb, H, K, 2), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    quant = ops.kv_quant("int4", k_token_scales=ks, v_token_scales=vs)
    g = torch.Generator().manual_seed(3)
    T = 40
    k, v = (torch.randn((T, H, D), generator=g).to(torch.bfloat16) for _ in range(2))
    blocks = [nb - 1, nb - 17, nb - 3]
    slots = torch.tensor([blocks[t // K] * K + t % K for t in range(T)], device=DEV)
    ops.paged_kv_write_quant(k.to(DEV), v.to(DEV), slots, kc, vc, quant)
    bt = torch.tensor([blocks], dtype=torch.int32, device=DEV)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 32, D), generator=g).to(torch.bfloat16)
    zero = np.zeros((3, K, H, D // 2), np.uint8), np.zeros((3, H, K, 2), np.uint16)
    pools = Q.kv_write_int4(zero[0], zero[0], zero[1], zero[1], k.float().numpy(), v.float().numpy(), range(T))
    ref = Q.paged_attention_decode_int4(storage(q), *pools, np.array([[0, 1, 2]]), [T], 0.1, "bf16")
    for kernel in (1, 2):
        out = ops.paged_attention_decode_quant(q.to(DEV), kc, vc, bt, lens, 0.1, quant, max_context_len=T,
                                               kernel=kernel)
        check_attention(as_f64(out), ref, "bf16")
    # the partly filled third block to another, and the attention through the copy
    pairs = torch.tensor([[blocks[2], nb - 30]], device=DEV)
    ops.kv_fork_copy(kc, vc, pairs, lens, quant=quant)
    bt[0, 2] = nb - 30
    out = ops.paged_attention_decode_quant(q.to(DEV), kc, vc, bt, lens, 0.1, quant, max_context_len=T)
    check_attention(as_f64(out), ref, "bf16")
    assert ops.get_device_error() == 0


def test_logits_past_32_bits(ops):
    # rows more than 2^31 values apart
    V, B = 5000, 2
    wide = torch.empty((2, 2**31 + 64), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(4)
    logits = (torch.randn((2, V), generator=g) * 3).to(torch.bfloat16)
    view = wide[:, 64:64 + V]
    view.copy_(logits)
    scores = torch.tensor([[-1.0, -1.5]])
    t, p, s, f = ops.beam_select(view, scores.to(DEV), 6)
    wt, wp, _, _ = OB.beam_select(logits.double().numpy(), scores.double().numpy(), 6)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(p.cpu().numpy(), wp)


def test_many_sequences(ops):
    # more sequences than one launch takes, with and without groups
    from tests.test_gpu_int4 import check, make
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    c = make(lens, 4, 2, 128, 16, torch.bfloat16, seed=1, share=1, group=4)
    check(ops, c, 0.1)
    check(ops, c, 0.1, share_prefix=True)


def test_long_rows_of_few_sequences(ops):
    # many partials a row: merged by a CTA a row
    from tests.test_gpu_int4 import check, make
    for lens in ([9000], [4000, 12000], [1, 20000, 7]):
        c = make(lens, 8, 4, 128, 16, torch.bfloat16, seed=sum(lens))
        a = check(ops, c, 128 ** -0.5)
        assert torch.equal(a, check(ops, c, 128 ** -0.5))


def test_workspace_too_small_is_refused(ops):
    from tests.test_gpu_int4 import make, on_gpu
    g = on_gpu(ops, make([300, 5], 8, 4, 128, 16, torch.bfloat16, seed=1))
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(ops.PagedKVError):
        ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=300, workspace=small)
    with pytest.raises(ops.PagedKVError):
        ops.beam_select(torch.zeros((8, 4000), device=DEV), torch.zeros((2, 4), device=DEV), 4, workspace=small)


def test_binding_refusals(ops):
    i32 = torch.int32
    logits, scores = torch.zeros((4, 50), device=DEV), torch.zeros((2, 2), device=DEV)
    with pytest.raises(ValueError):
        ops.beam_select(logits[:3], scores, 2)
    with pytest.raises(ValueError):
        ops.beam_select(logits.t().contiguous().t(), scores, 2)
    with pytest.raises(TypeError):
        ops.beam_select(logits.half(), scores, 2)
    with pytest.raises(TypeError):
        ops.beam_select(logits, scores, 2, finished=torch.zeros((2, 2), device=DEV), eos_token=1)
    with pytest.raises(ops.PagedKVError):
        ops.beam_select(logits, scores, 2, finished=torch.zeros((2, 2), dtype=torch.bool, device=DEV))
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device=DEV)
    ks = torch.zeros((4, 2, 16, 2), dtype=torch.bfloat16, device=DEV)
    qd = ops.kv_quant("int4", k_token_scales=ks, v_token_scales=ks.clone())
    k = torch.zeros((3, 2, 128), device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        ops.paged_kv_write_quant(k, k, slots, kc[:3], kc[:3], qd)            # scales of another pool
    with pytest.raises(ValueError):
        ops.paged_kv_write_quant(k[:, :, :64], k, slots, kc, kc.clone(), qd)
    with pytest.raises(TypeError):
        ops.paged_kv_write_quant(k, k, slots.to(i32), kc, kc.clone(), qd)
    with pytest.raises(ValueError):
        ops.paged_kv_write_quant(k, k, slots, kc.cpu(), kc, qd)
    with pytest.raises(ValueError):
        ops.paged_qk_norm_rope_append(k, k, k, slots.to(i32), slots, kc, kc.clone(),
                                      torch.zeros((4, 0), device=DEV), quant=qd)
    parents = torch.zeros((2, 2), dtype=i32, device=DEV)
    v4 = torch.zeros(4, dtype=i32, device=DEV)
    tables = torch.zeros((4, 3), dtype=i32, device=DEV)
    ring, state = torch.zeros(8, dtype=i32, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        ops.fork_tables(parents, v4[:3], v4, tables, ring, state, 16)
    with pytest.raises(ValueError):
        ops.fork_tables(parents, v4, v4, tables[:, :2], ring, state, 16)
    with pytest.raises(TypeError):
        ops.fork_tables(parents.long(), v4, v4, tables, ring, state, 16)
    with pytest.raises(ValueError):
        ops.kv_fork_copy(kc, kc.clone(), torch.zeros((3, 2), dtype=torch.int64, device=DEV), v4, quant=qd)


@pytest.mark.parametrize("H_q,H_kv,K,group,share,splits", [(16, 16, 16, 8, 30, 5), (32, 8, 16, 8, 7, 8), (16, 8, 16, 4, 20, 5)])
def test_warps_that_lag(ops, H_q, H_kv, K, group, share, splits):
    # empty sequences: the warp that zeroes their rows starts late on its tiles; every
    # call gives the same bits
    from tests.test_gpu_int4 import check, make, on_gpu
    rng = np.random.default_rng(H_q + K)
    lens = [int(x) for x in rng.integers(1, 400, 3 * group + 1)]
    for z in (0, 1, 6, 7):
        lens[z] = 0
    c = make(lens, H_q, H_kv, 128, K, torch.bfloat16, seed=share, share=share, group=group)
    want = check(ops, c, 0.1, share_prefix=True, kernel=1, num_splits=splits)
    g = on_gpu(ops, c)
    for _ in range(500):
        assert torch.equal(want, ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=max(lens),
                                                                  share_prefix=True, kernel=1, num_splits=splits))


def test_one_row_forked_to_all(ops):
    # the same parent for every row of a group, one workspace used by two captured graphs in turn
    i32 = torch.int32
    R, B, K, W = 2, 8, 4, 5
    tables = torch.arange(R * B * W, dtype=i32, device=DEV).view(R * B, W)
    held = torch.full((R * B,), W, dtype=i32, device=DEV)
    lens = torch.full((R * B,), W * K - 1, dtype=i32, device=DEV)
    ring = torch.full((128,), -1, dtype=i32, device=DEV)
    ring[:32] = torch.arange(100, 132, dtype=i32, device=DEV)
    state = torch.tensor([0, 32], dtype=torch.int64, device=DEV)
    parents = torch.tensor([[3] * B, [0] * B], dtype=i32, device=DEV)
    ws = torch.empty(ops.fork_workspace_bytes(R, B, W), dtype=torch.uint8, device=DEV)
    outs = [dict(block_tables_out=tables.clone(), lens_out=lens.clone(), held_out=held.clone(),
                 ring_state_out=state.clone(), pairs=torch.empty((R * B, 2), dtype=torch.int64, device=DEV),
                 totals=torch.empty(4, dtype=i32, device=DEV), ring=ring.clone()) for _ in range(2)]

    def run(o):
        o = dict(o)
        r = o.pop("ring")
        ops.fork_tables(parents, lens, held, tables, r, state, K, workspace=ws, **o)

    run(outs[0])                                              # (loads every kernel)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run(o)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    a, b = outs
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert a["totals"].tolist()[0] == 0
    t = a["block_tables_out"].cpu().numpy().reshape(R, B, W)
    keep = [3, 0]
    for r in range(R):
        src = tables.cpu().numpy().reshape(R, B, W)[r, keep[r]]
        assert (t[r, :, :W - 1] == src[:W - 1]).all()          # whole blocks shared
        assert len(set(t[r, :, W - 1].tolist())) == B           # a tail each
    s0, s1 = a["ring_state_out"].tolist()
    rg = a["ring"].cpu().numpy()
    free = [int(rg[j % len(rg)]) for j in range(s0, s1)]
    assert sorted(free + sorted(set(t.reshape(-1).tolist()))) == list(range(R * B * W)) + list(range(100, 132))
