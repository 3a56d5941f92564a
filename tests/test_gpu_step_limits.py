"""The step calls at their edges: one directly behind the other on lengths that
the kernel in front writes, two at once, captured, pools past 32-bit offsets,
running counts past 32 bits, rows too wide for the ring of stages."""

import numpy as np
import pytest
import torch

from oracle import step as O
from tests._helpers import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def test_attention_right_behind_the_tables(ops):
    """Lengths, tables and slots are read by the next kernels without a host
    wait in between, while the one that writes them may still run."""
    S, H, J, D, K = 40, 16, 4, 128, 16
    shared, width, nb = 6, 14, 400
    rng = np.random.default_rng(0)
    g = torch.Generator().manual_seed(0)
    order = rng.permutation(nb).astype(np.int32)
    kc, vc = (torch.randn((nb, K, J, D), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn((S, H, D), generator=g).to(torch.bfloat16).to(DEV)
    kv = torch.randn((S, J, D), generator=g).to(torch.bfloat16).to(DEV)
    table = i32(order[:shared])
    want = None
    for it in range(30):
        tables = np.full((S, width), -1, np.int32)
        tables[:, :shared] = order[:shared]
        t, held = i32(tables), i32([shared] * S)
        lens = i32([shared * K] * S)
        ctx = torch.full((S,), -5, dtype=torch.int32, device=DEV)      # what a reader too early sees
        torch.cuda.synchronize()
        o = ops.step_tables(lens, i32([1] * S), t, held, i32(order),
                            torch.tensor([shared, nb], device=DEV), K, nb, num_tokens=S,
                            context_lens=ctx)
        if it % 2:
            ops.paged_kv_write(kv, kv, o["slots"], kc, vc)
        out = ops.paged_attention_decode_prefix(q, kc, vc, table, t, ctx, D ** -0.5,
                                                prefix_len=shared * K, max_context_len=200) \
            if it % 4 < 2 else ops.paged_attention_decode(q, kc, vc, t, ctx, D ** -0.5,
                                                          max_context_len=200)
        if it == 1:
            want = out.clone()
        if it > 1:
            tol = 2.0**-6 * (1 + want.double().abs())
            assert bool(((out.double() - want.double()).abs() <= tol).all())
    assert ops.get_device_error() == 0


def test_two_at_once(ops):
    """The same calls on two streams, each with its own workspace and outputs."""
    S, H, J, D, K, P = 30, 32, 8, 128, 16, 1024
    g = torch.Generator(device=DEV).manual_seed(3)
    nb = P // K + 2 * S
    kc, vc = (torch.empty((nb, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
              for _ in range(2))
    rows = torch.cat([torch.arange(P // K, device=DEV)[None].expand(S, -1),
                      P // K + torch.arange(2 * S, device=DEV).view(S, 2)], 1).int().contiguous()
    lens = (P + torch.randint(1, 32, (S,), generator=g, device=DEV)).int()
    qs = [torch.randn((S, H, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    probs = [torch.softmax(3 * torch.randn((S, 50000), generator=g, device=DEV), -1) for _ in range(2)]
    tokens = torch.zeros(S, dtype=torch.int32, device=DEV)
    u = torch.rand(S, generator=g, device=DEV)
    cu = torch.arange(S + 1, device=DEV).int()

    def go(i):
        a = ops.paged_attention_decode_prefix(qs[i], kc, vc, rows[0].contiguous(), rows, lens,
                                              D ** -0.5, prefix_len=P, max_context_len=P + 32)
        return a, ops.verify_draft_tokens(probs[i], None, tokens, u, cu, 1)[0]
    ref = [go(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = go(i)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i][0], ref[i][0]) and torch.equal(got[i][1], ref[i][1])
    assert ops.get_device_error() == 0


def test_verification_captured(ops):
    S, V = 5, 3001
    g = torch.Generator(device=DEV).manual_seed(1)
    target = torch.softmax(2 * torch.randn((2 * S, V), generator=g, device=DEV), -1)
    draft = torch.softmax(2 * torch.randn((S, 1, V), generator=g, device=DEV), -1)
    tokens = torch.randint(0, V, (2 * S,), generator=g, device=DEV).int()
    u = torch.rand(2 * S, generator=g, device=DEV)
    cu = (2 * torch.arange(S + 1, device=DEV)).int()
    out, new = ops.verify_draft_tokens(target, draft, tokens, u, cu, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.verify_draft_tokens(target, draft, tokens, u, cu, 2, out_tokens=out, num_new=new)
    for _ in range(3):
        u.copy_(torch.rand(2 * S, generator=g, device=DEV))
        out.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        o, n = O.verify(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(),
                        u.cpu().numpy(), cu.cpu().numpy(), 2)
        assert np.array_equal(out.cpu().numpy(), o) and np.array_equal(new.cpu().numpy(), n)


def test_more_token_rows_than_the_sequences_can_have(ops):
    """A captured step's host bound on the rows may be far above what is used."""
    H, J, D, K = 4, 2, 64, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    kc, vc = (torch.empty((8, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
              for _ in range(2))
    rows = torch.arange(8, device=DEV).int().view(1, 8)
    q = torch.randn((64, H, D), generator=g, device=DEV).to(torch.bfloat16)
    cu, lens = i32([0, 2]), i32([100])
    kw = dict(prefix_len=64, max_context_len=128, cu_seqlens=cu, max_query_len=2)
    out = torch.full_like(q, 3.0)
    ops.paged_attention_decode_prefix(q, kc, vc, rows[0], rows, lens, 0.1, out=out, **kw)
    ref = ops.paged_attention_decode_prefix(q[:2].contiguous(), kc, vc, rows[0], rows, lens, 0.1, **kw)
    assert ops.get_device_error() == 0
    assert (out[2:] == 3.0).all()
    assert bool(((out[:2].double() - ref.double()).abs() <= 2.0**-6 * (1 + ref.double().abs())).all())


def test_pools_past_32_bit_offsets(ops):
    """Pools of more than 2^31 values: pages at their end, written by the
    rotation and read by the attention."""
    J, D, K, H = 8, 128, 16, 16
    nb = 2**31 // (J * D * K) + 64
    kc, vc = (torch.zeros((nb, K, J, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(4)
    n = 4 * K                                          # four blocks at the pool's end
    qkv = torch.randn((n, H + 2 * J, D), generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.arange(nb * K - n, nb * K, device=DEV)
    table = torch.zeros((32, D), device=DEV)
    table[:, :D // 2] = 1                              # no turn: the rows as they are
    pos = (torch.arange(n, device=DEV) % 32).int()
    ops.paged_qk_norm_rope_append(qkv[:, :H], qkv[:, H:H + J], qkv[:, H + J:], pos, slots, kc, vc,
                                  table)
    assert torch.equal(kc.view(-1, J, D)[slots], qkv[:, H:H + J])
    assert torch.equal(vc.view(-1, J, D)[slots], qkv[:, H + J:])
    assert not kc.view(-1, J, D)[nb * K - n - 64:nb * K - n].any()
    rows = torch.arange(nb - 4, nb, device=DEV).int().view(1, 4)
    q = qkv[:1, :H].contiguous()
    got = ops.paged_attention_decode_prefix(q, kc, vc, rows[0, :2].contiguous(), rows, i32([n - 3]),
                                            0.1, prefix_len=2 * K, max_context_len=n)
    k, v = (x[:n - 3].double().repeat_interleave(H // J, 1) for x in (qkv[:, H:H + J], qkv[:, H + J:]))
    w = torch.softmax(torch.einsum("hd,xhd->hx", q[0].double(), k) * 0.1, -1)
    ref, a = torch.einsum("hx,xhd->hd", w, v), torch.einsum("hx,xhd->hd", w, v.abs())
    assert bool(((got[0].double() - ref).abs() <= (2.0**-7 + 2.0**-8) * a + 2.0**-8 * ref.abs()).all())
    assert ops.get_device_error() == 0


def test_running_counts_past_32_bits(ops):
    R = 50
    head = 2**40 + 13
    ring = np.arange(R, dtype=np.int32)[::-1].copy()
    tables = np.full((3, 20), -1, np.int32)
    tables[2, :5] = [40, 41, 42, 43, 44]
    args = ([0, 0, 17], [30, 7, -1], tables, [0, 0, 5], None, ring, [head, head + 30])
    want = O.step_tables(*args, 4, 64)
    t, r = i32(tables), i32(ring)
    o = ops.step_tables(i32(args[0]), i32(args[1]), t, i32(args[3]), r,
                        torch.tensor(args[6], device=DEV), 4, 50, num_tokens=64)
    assert want["totals"][0] == 0 == ops.get_device_error()
    assert np.array_equal(t.cpu().numpy(), want["tables"])
    assert np.array_equal(r.cpu().numpy(), want["ring"])
    assert o["ring_state_out"].tolist() == want["state"]
    assert np.array_equal(o["slots"].cpu().numpy(), want["slots"])


@pytest.mark.parametrize("fmt", [None, "fp8"])
def test_rows_too_wide_for_the_ring(ops, fmt):
    """Two stages of a token of 440 heads do not fit shared memory."""
    T, H, J, D, K = 3, 424, 8, 128, 4
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((T, H + 2 * J, D), generator=g).to(torch.bfloat16)
    ang = np.arange(9)[:, None] * (10000.0 ** (-np.arange(0, D, 2) / D))[None]
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    d = qkv.to(DEV)
    dt = torch.bfloat16 if fmt is None else torch.uint8
    kc, vc = (torch.zeros((2, K, J, D), dtype=dt, device=DEV) for _ in range(2))
    quant = None if fmt is None else ops.kv_quant(fmt, 0.03125, 0.03125)
    out = ops.paged_qk_norm_rope_append(d[:, :H], d[:, H:H + J], d[:, H + J:], i32([8, 0, 3]),
                                        torch.tensor([7, 2, 5], device=DEV), kc, vc,
                                        torch.from_numpy(table).to(DEV), quant=quant)
    assert ops.get_device_error() == 0
    x = as_f64(qkv)
    for t, p in enumerate([8, 0, 3]):
        for h in range(0, H, 53):
            ref = O.norm_rope(x[t, h], None, 0.0, p, table)
            pair = np.hypot(x[t, h], np.roll(x[t, h], D // 2)) * 2**0.5
            assert np.all(np.abs(as_f64(out[t, h]) - ref) <= 2.0**-8 * np.abs(ref) + 4 * 2.0**-24 * pair)
    if fmt is None:
        assert torch.equal(vc.view(-1, J, D)[[7, 2, 5]].cpu(), qkv[:, H + J:])
