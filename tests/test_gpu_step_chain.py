"""Speculative decoding steps behind a shared prompt, the calls one after the
other as an engine makes them: step tables from lengths, head norms + rotation
+ append, attention behind the shared prefix, draft verification, and the
accepted counts into the next step's lengths, with no host read in between.

The model around them is random: its projection's rows and its probabilities
come from a seed.  Checked per step: tables, slots and accepted tokens equal
oracle/step.py; the pages' rows and the queries within the rotation's bound;
the attention within its bound, from the pages as they are on the GPU.
"""

import numpy as np
import pytest
import torch

from oracle import prefill as P
from oracle import step as O
from tests._helpers import as_f64, storage

pytestmark = pytest.mark.gpu

DEV = "cuda"
S, H, J, D, K, V = 6, 8, 4, 64, 8, 97
PREFIX, ROWS, WIDTH, BLOCKS, STEPS = 40, 4, 14, 64, 5
T = S * ROWS                                   # host bound on the tokens of a step


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Engine:
    def __init__(self, ops):
        self.ops = ops
        rng = np.random.default_rng(0)
        order = rng.permutation(BLOCKS).astype(np.int32)
        n = PREFIX // K
        tables = np.full((S, WIDTH), -1, np.int32)
        tables[:, :n] = order[:n]
        self.table = i32(order[:n])
        self.tables, self.ring = i32(tables), i32(order)
        self.state = torch.tensor([n, BLOCKS], dtype=torch.int64, device=DEV)
        self.lens, self.held = i32([PREFIX] * S), i32([n] * S)
        self.shared, self.counts = i32([n] * S), i32([1] * S)
        g = torch.Generator().manual_seed(1)
        self.kc = torch.randn((BLOCKS, K, J, D), generator=g).to(torch.bfloat16).to(DEV)
        self.vc = torch.randn((BLOCKS, K, J, D), generator=g).to(torch.bfloat16).to(DEV)
        ang = np.arange(WIDTH * K)[:, None] * (10000.0 ** (-np.arange(0, D, 2) / D))[None]
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().to(DEV)
        self.wq = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
        self.wk = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
        # a step's inputs, in place so that a captured step reads them
        self.qkv = torch.zeros((T, (H + 2 * J) * D), dtype=torch.bfloat16, device=DEV)
        self.target = torch.zeros((T, V), device=DEV)
        self.draft = torch.zeros((S, ROWS - 1, V), device=DEV)
        self.tokens = torch.zeros(T, dtype=torch.int32, device=DEV)
        self.uniforms = torch.zeros(T, device=DEV)
        self.out = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
        self.q_out = torch.zeros_like(self.out)
        self.ws = torch.empty(max(256, ops.prefix_workspace_bytes(
            S, T, ROWS, WIDTH * K, PREFIX, H, J, D, K, torch.bfloat16)), dtype=torch.uint8,
            device=DEV)
        self.step_out = None

    def step(self):
        ops, f = self.ops, self.qkv.unflatten(1, (H + 2 * J, D))
        self.step_out = ops.step_tables(self.lens, self.counts, self.tables, self.held, self.ring,
                                        self.state, K, BLOCKS, shared=self.shared, num_tokens=T,
                                        held_out=self.held, ring_state_out=self.state,
                                        **({k: self.step_out[k] for k in
                                            ("context_lens", "cu_seqlens", "cu_blocks",
                                             "positions", "slots", "totals")}
                                           if self.step_out else {}))
        o = self.step_out
        ops.paged_qk_norm_rope_append(f[:, :H], f[:, H:H + J], f[:, H + J:], o["positions"],
                                      o["slots"], self.kc, self.vc, self.cos_sin, self.wq,
                                      self.wk, q_out=self.q_out)
        ops.paged_attention_decode_prefix(self.q_out, self.kc, self.vc, self.table, self.tables,
                                          o["context_lens"], D ** -0.5, prefix_len=PREFIX,
                                          max_context_len=WIDTH * K, cu_seqlens=o["cu_seqlens"],
                                          max_query_len=ROWS, out=self.out, workspace=self.ws)
        self.verified = ops.verify_draft_tokens(self.target, self.draft, self.tokens,
                                                self.uniforms, o["cu_seqlens"], ROWS)
        self.lens.add_(self.verified[1])       # the accepted rows stay in the cache
        self.lens.mul_(self.counts >= 0)

    def inputs(self, it):
        """New random inputs of step `it`, written in place; host copies."""
        rng = np.random.default_rng(100 + it)
        g = torch.Generator().manual_seed(100 + it)
        counts = rng.integers(1, ROWS + 1, S)
        if it == 3:
            counts[2] = -1                     # over: its own blocks come back
        if it == 4:
            counts[2] = 0
        self.counts.copy_(i32(counts))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).to(torch.bfloat16))
        p = torch.softmax(2 * torch.randn((T, V), generator=g), -1)
        self.target.copy_(p)
        d = torch.softmax(2 * torch.randn((S, ROWS - 1, V), generator=g), -1)
        cu = np.concatenate([[0], np.cumsum(np.maximum(counts, 0))])
        for s in range(S):                     # drafts near the target: some are accepted
            for i in range(max(int(counts[s]) - 1, 0)):
                d[s, i] = 0.5 * d[s, i] + 0.5 * p[cu[s] + i]
        self.draft.copy_(d)
        tokens = rng.integers(0, V, T)
        for s in range(S):
            for i in range(max(int(counts[s]) - 1, 0)):
                tokens[cu[s] + i + 1] = int(torch.multinomial(d[s, i], 1, generator=g))
        self.tokens.copy_(i32(tokens))
        self.uniforms.copy_(torch.rand(T, generator=g))
        return counts, tokens

    def check(self, before, counts, tokens):
        o = {k: v.cpu().numpy() for k, v in self.step_out.items()}
        w = O.step_tables(before["lens"], counts, before["tables"], before["held"],
                          [PREFIX // K] * S, before["ring"], before["state"], K, T)
        assert w["totals"][0] == 0 == o["totals"][0]
        assert np.array_equal(self.tables.cpu().numpy(), w["tables"])
        assert np.array_equal(self.ring.cpu().numpy(), w["ring"])
        assert np.array_equal(o["slots"], w["slots"])
        assert list(o["cu_seqlens"]) == w["cu_seqlens"]
        assert list(o["context_lens"]) == w["context_lens"]
        cu, n = w["cu_seqlens"], w["cu_seqlens"][-1]
        # queries and pages: float32 up to one rounding to bf16
        rows = as_f64(self.qkv).reshape(T, H + 2 * J, D)
        table = as_f64(self.cos_sin)
        kc = as_f64(self.kc).reshape(-1, J, D)
        for t in range(n):
            for h in range(H + J):
                ref = O.norm_rope(rows[t, h], as_f64(self.wq if h < H else self.wk), 1e-6,
                                  int(o["positions"][t]), table)
                got = as_f64(self.q_out[t, h]) if h < H else kc[o["slots"][t], h - H]
                pair = np.hypot(ref, np.roll(ref, D // 2)) * 2**0.5     # >= |a| + |b|
                assert np.all(np.abs(got - ref) <= 2.0**-8 * np.abs(ref) + 25 * 2.0**-24 * pair)
            assert torch.equal(self.vc.view(-1, J, D)[int(o["slots"][t])],
                               self.qkv.unflatten(1, (H + 2 * J, D))[t, H + J:])
        live = [s for s in range(S) if counts[s] > 0]
        lens = [w["context_lens"][s] for s in live]
        c2 = np.concatenate([[0], np.cumsum([counts[s] for s in live])])
        args = (storage(self.q_out[:n]), storage(self.kc))
        ref, a = (P.paged_attention_prefill(*args, storage(v), w["tables"][live], c2, lens,
                                            D ** -0.5, "bf16") for v in (self.vc, self.vc.abs()))
        err = np.abs(as_f64(self.out[:n]) - ref)
        assert np.all(err <= (2.0**-7 + 2.0**-8) * a + 2.0**-8 * np.abs(ref))
        out, new = O.verify(self.target.cpu().numpy(), self.draft.cpu().numpy(), tokens,
                            self.uniforms.cpu().numpy(), cu, ROWS)
        assert np.array_equal(self.verified[0].cpu().numpy(), out)
        assert np.array_equal(self.verified[1].cpu().numpy(), new)
        lens = [0 if counts[s] < 0 else before["lens"][s] + int(new[s]) for s in range(S)]
        assert self.lens.cpu().tolist() == lens
        return new

    def now(self):
        return dict(lens=self.lens.cpu().tolist(), tables=self.tables.cpu().numpy(),
                    held=self.held.cpu().tolist(), ring=self.ring.cpu().numpy(),
                    state=self.state.cpu().tolist())


@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps(ops, captured):
    e = Engine(ops)
    accepted = 0
    graph = None
    for it in range(STEPS):
        before = e.now()
        counts, tokens = e.inputs(it)
        if captured and it == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                e.step()
        if graph is not None:
            graph.replay()
        else:
            e.step()
        torch.cuda.synchronize()
        assert ops.get_device_error() == 0
        accepted += int((e.check(before, counts, tokens) > 1).sum())
    assert accepted > 0 and int(e.state[1]) > BLOCKS       # drafts accepted, blocks came back
