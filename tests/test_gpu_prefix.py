"""GPU parity of attention behind a shared prefix against the float64 oracle.

Tolerance.  The weights of the softmax enter the tensor cores rounded to
bf16 (half a step: 2^-8 relative); the sum that divides them is that of the
weights before or after the rounding, so the output is off by at most 2 * 2^-8
of A = sum_x w_x |v_x| (the attention over |V|), the store rounds by 2^-8 of
the value.  A score is a float32 sum of D <= 128 products; scores stay below
2^9 in magnitude (base 2), so that a weight is off by less than 128 * 2^-24 *
2^9 = 2^-8 through it: 2^-8 of A more.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import prefill as P
from tests._helpers import as_f64, storage

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def problem(lens, news, H, J, D, K, prefix, seed=0, spread=1.0):
    """Sequences of lens[s] tokens (news[s] of them new) that share their
    first `prefix` tokens.  Unused slots hold NaN, unused entries garbage."""
    rng = np.random.default_rng(seed)
    S, shared = len(lens), prefix // K
    blocks = [max(0, -(-L // K) - shared) for L in lens]
    nb = shared + sum(blocks) + 3
    order = rng.permutation(nb)
    width = max([-(-L // K) for L in lens] + [shared, 1]) + 2
    bt = rng.integers(-5, nb + 50, size=(S, width)).astype(np.int32)
    full = bt.copy()                                 # what the oracle reads
    at = shared
    live = np.zeros(nb * K, bool)
    for s, L in enumerate(lens):
        full[s, :shared] = order[:shared]
        full[s, shared:shared + blocks[s]] = order[at:at + blocks[s]]
        bt[s, shared:] = full[s, shared:]            # prefix entries stay garbage: never read
        at += blocks[s]
        for x in range(L):
            live[full[s, x // K] * K + x % K] = True
    for x in range(prefix):
        live[order[x // K] * K + x % K] = True
    g = torch.Generator().manual_seed(seed)
    kc = (torch.randn((nb, K, J, D), generator=g) * spread).to(torch.bfloat16)
    vc = torch.randn((nb, K, J, D), generator=g).to(torch.bfloat16)
    dead = torch.from_numpy(~live.reshape(nb, K))
    kc[dead] = float("nan")
    vc[dead] = float("nan")
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = torch.randn((int(cu[-1]), H, D), generator=g).to(torch.bfloat16)
    return dict(lens=list(lens), cu=cu, bt=bt, full=full, kc=kc, vc=vc, q=q, K=K, prefix=prefix,
                table=order[:shared].astype(np.int32), scale=D ** -0.5, most=max(lens),
                max_q=max(list(news) + [1]), single=all(n == 1 for n in news))


def call(ops, pb, cu=None, out=None, **kw):
    use = pb["cu"] if cu is None and not pb["single"] else cu
    return ops.paged_attention_decode_prefix(
        pb["q"].to(DEV), pb["kc"].to(DEV), pb["vc"].to(DEV), torch.from_numpy(pb["table"]).to(DEV),
        torch.from_numpy(pb["bt"]).to(DEV),
        torch.tensor(pb["lens"], dtype=torch.int32, device=DEV), pb["scale"],
        prefix_len=pb["prefix"], max_context_len=pb["most"],
        cu_seqlens=None if use is None else torch.from_numpy(use).to(DEV),
        max_query_len=pb["max_q"] if use is not None else 1, out=out, **kw)


def want(pb):
    def att(v):
        if pb["single"]:
            return oracle.paged_attention_decode(storage(pb["q"]), storage(pb["kc"]), storage(v),
                                                 pb["full"], pb["lens"], pb["scale"], "bf16")
        return P.paged_attention_prefill(storage(pb["q"]), storage(pb["kc"]), storage(v),
                                         pb["full"], pb["cu"], pb["lens"], pb["scale"], "bf16")
    return att(pb["vc"]), att(pb["vc"].abs())


def check(ops, pb, got=None):
    got = as_f64(call(ops, pb) if got is None else got)
    assert ops.get_device_error() == 0
    ref, a = want(pb)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    tol = (2.0**-7 + 2.0**-8) * a + 2.0**-8 * np.abs(ref)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("H,J,D", [(8, 8, 128), (8, 2, 128), (8, 1, 64), (14, 2, 128), (16, 2, 64),
                                   (6, 3, 128)])
@pytest.mark.parametrize("K", [8, 16, 48])
def test_heads_and_blocks(ops, H, J, D, K):
    rng = np.random.default_rng(H + K)
    prefix = 5 * K
    lens = [prefix + int(x) for x in rng.integers(1, 200, 7)]
    check(ops, problem(lens, [1] * 7, H, J, D, K, prefix, seed=K))


@pytest.mark.parametrize("prefix", [0, 16, 64, 112, 128, 144, 1040, 4096])
def test_prefix_lengths(ops, prefix):
    lens = [prefix + x for x in (1, 2, 16, 17, 63, 64, 65, 300)]
    check(ops, problem(lens, [1] * 8, 8, 2, 128, 16, prefix, seed=prefix))


@pytest.mark.parametrize("S", [1, 2, 31, 33, 64, 65, 129, 300])
def test_batch_sizes(ops, S):
    """Query rows of one KV head that end anywhere in a tile of 128 rows, in
    one tile, two, or several."""
    rng = np.random.default_rng(S)
    lens = [160 + int(x) for x in rng.integers(1, 50, S)]
    check(ops, problem(lens, [1] * S, 4, 1, 128, 16, 160, seed=S))


def test_sequences_at_and_below_the_prefix(ops):
    """Lengths that end inside the prefix, at its end, and empty sequences."""
    lens = [0, 1, 7, 64, 65, 127, 128, 129, 0, 200, 192, 191]
    pb = problem(lens, [1] * len(lens), 8, 2, 128, 16, 192, seed=3)
    out = call(ops, pb)
    assert (out[0] == 0).all() and (out[8] == 0).all()
    check(ops, pb, out)


@pytest.mark.parametrize("H,J,most", [(8, 8, 8), (16, 8, 4), (8, 2, 2), (12, 4, 2)])
def test_packed_new_tokens(ops, H, J, most):
    rng = np.random.default_rng(H)
    news = [int(x) for x in rng.integers(1, most + 1, 23)]
    lens = [224 + n + int(x) for n, x in zip(news, rng.integers(0, 90, 23))]
    check(ops, problem(lens, news, H, J, 128, 16, 224, seed=H))


@pytest.mark.parametrize("H,J,D,K", [(32, 16, 128, 16), (12, 12, 64, 8), (48, 24, 64, 32),
                                     (10, 10, 128, 16)])
def test_several_groups_of_kv_heads(ops, H, J, D, K):
    """More KV heads than the decode kernel takes in one CTA."""
    rng = np.random.default_rng(J)
    lens = [6 * K + int(x) for x in rng.integers(1, 120, 9)]
    check(ops, problem(lens, [1] * 9, H, J, D, K, 6 * K, seed=J))
    news = [int(x) for x in rng.integers(1, 3, 9)]
    check(ops, problem(lens, news, H, J, D, K, 6 * K, seed=J + 1))


def test_the_largest_batch(ops):
    """2048 sequences, the most of one call, most of them a token or two behind
    the prefix."""
    rng = np.random.default_rng(7)
    lens = [int(x) for x in 64 + rng.integers(1, 4, 2048)]
    lens[5], lens[2000] = 0, 40
    pb = problem(lens, [1] * 2048, 2, 1, 64, 16, 64, seed=7)
    check(ops, pb)
    with pytest.raises(ops.PagedKVError):
        call(ops, dict(pb, lens=lens + [1], q=torch.cat([pb["q"], pb["q"][:1]]),
                       bt=np.concatenate([pb["bt"], pb["bt"][:1]])))


def test_packed_new_tokens_inside_the_prefix(ops):
    """New tokens that sit in shared blocks see the keys up to their own."""
    news = [4, 4, 2, 1, 4]
    lens = [162, 160, 80, 5, 4]
    check(ops, problem(lens, news, 16, 8, 128, 16, 160, seed=8))


def test_sequences_without_new_tokens_and_rows_behind(ops):
    news = [2, 0, 3, 0, 1]
    lens = [100, 90, 120, 80, 81]
    pb = problem(lens, news, 4, 2, 64, 16, 80, seed=9)
    ref = call(ops, pb)
    check(ops, pb, ref)
    wide = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    pb2 = dict(pb, q=torch.cat([pb["q"], torch.randn(3, 4, 64).to(torch.bfloat16)]))
    call(ops, pb2, out=wide)
    assert torch.equal(wide[:6], ref) and (wide[6:] == 5.0).all()
    assert ops.get_device_error() == 0


def test_sharp_and_flat_scores(ops):
    """Scores that differ by hundreds (one key takes all), and equal ones."""
    pb = problem([700, 513, 600], [1, 1, 1], 8, 2, 128, 16, 512, seed=4, spread=40.0)
    check(ops, pb)
    pb = problem([700, 513, 600], [1, 1, 1], 8, 2, 128, 16, 512, seed=4)
    pb["q"].zero_()
    check(ops, pb)
    # the largest score late: the running maximum rises in every tile
    pb = problem([300] * 5, [1] * 5, 4, 1, 128, 16, 288, seed=5)
    ramp = torch.linspace(0, 6, pb["table"].size * 16).view(-1, 16, 1, 1)
    pb["kc"][torch.from_numpy(pb["table"]).long()] = (pb["q"][0, 0].float() * ramp).to(torch.bfloat16)
    check(ops, pb)


def test_equals_attention_over_the_full_tables(ops):
    """The framework's own decode call over the full rows, within both bounds."""
    pb = problem([1000 + 7 * i for i in range(20)], [1] * 20, 32, 8, 128, 16, 960, seed=6)
    got = as_f64(call(ops, pb))
    ref = as_f64(ops.paged_attention_decode(
        pb["q"].to(DEV), pb["kc"].to(DEV), pb["vc"].to(DEV), torch.from_numpy(pb["full"]).to(DEV),
        torch.tensor(pb["lens"], dtype=torch.int32, device=DEV), pb["scale"]))
    _, a = want(dict(pb, full=pb["full"]))
    assert np.all(np.abs(got - ref) <= 2.0**-6 * a + 2.0**-6 * np.abs(ref))


def test_bad_blocks_and_lengths_are_reported(ops):
    pb = problem([100, 120], [1, 1], 4, 2, 128, 16, 64, seed=2)
    bad = dict(pb, bt=pb["bt"].copy())
    bad["bt"][1, 5] = 10**6
    call(ops, bad)
    assert ops.get_device_error() == 1
    bad = dict(pb, table=pb["table"].copy())
    bad["table"][2] = -3
    call(ops, bad)
    assert ops.get_device_error() == 1
    call(ops, dict(pb, lens=[100, 10**6]))
    assert ops.get_device_error() == 4
    call(ops, dict(pb, lens=[-1, 120]))
    assert ops.get_device_error() == 4
    two = problem([100, 120], [2, 2], 4, 2, 128, 16, 64, seed=2)
    out = torch.full((4, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    ref = call(ops, two)
    call(ops, dict(two, lens=[1, 120]), out=out)               # two new tokens, one cached
    assert ops.get_device_error() == 4
    assert (out[:2] == 5.0).all() and torch.equal(out[2:], ref[2:])


def test_repeats_bit_for_bit_and_on_another_stream(ops):
    pb = problem([600 + 3 * i for i in range(40)], [1] * 40, 8, 2, 128, 16, 576, seed=1)
    a = call(ops, pb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(ops, pb)
    side.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("S,H,prefix", [(8, 64, 65536), (3, 8, 65536), (20, 64, 16384), (40, 64, 8192)])
def test_long_prefix_repeats_bit_for_bit(ops, S, H, prefix):
    """A prefix far larger than the caches, one to three tiles of query rows a
    KV head: waits for memory in every step, the same bits every time, and the
    framework's decode call over the full rows."""
    J, D, K = 8, 128, 32
    g = torch.Generator(device=DEV).manual_seed(prefix + S)
    own = 64
    shared, nb = prefix // K, prefix // K + S * 3
    kc, vc = (torch.empty((nb, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
              for _ in range(2))
    order = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    rows = torch.cat([order[:shared][None].expand(S, -1), order[shared:].view(S, 3)], 1).contiguous()
    lens = prefix + torch.randint(1, own, (S,), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randn((S, H, D), generator=g, device=DEV).to(torch.bfloat16)
    call = lambda: ops.paged_attention_decode_prefix(  # noqa: E731
        q, kc, vc, order[:shared].contiguous(), rows, lens, D ** -0.5, prefix_len=prefix,
        max_context_len=prefix + own)
    first = call()
    for _ in range(30):
        assert torch.equal(call().view(torch.int16), first.view(torch.int16))
    ref = ops.paged_attention_decode(q, kc, vc, rows, lens, D ** -0.5, max_context_len=prefix + own)
    a = ops.paged_attention_decode(q, kc, vc.abs(), rows, lens, D ** -0.5, max_context_len=prefix + own)
    assert ops.get_device_error() == 0
    err = (first.double() - ref.double()).abs()
    assert bool((err <= (2.0**-7 + 2.0**-8) * a.double() * (1 + 2.0**-8) + 2.0**-7 * ref.double().abs()).all())
    # the weights' roundings are independent: they add up like noise, not like the bound
    assert float(err.norm() / ref.double().norm()) < 4 * 2.0**-8


def test_captured_and_replayed(ops):
    pb = problem([400 + 3 * i for i in range(9)], [1] * 9, 8, 2, 128, 16, 384, seed=1)
    t = {k: pb[k].to(DEV) for k in ("q", "kc", "vc")}
    bt, table = torch.from_numpy(pb["bt"]).to(DEV), torch.from_numpy(pb["table"]).to(DEV)
    lens = torch.tensor(pb["lens"], dtype=torch.int32, device=DEV)
    outs = [torch.empty_like(t["q"]) for _ in range(2)]
    ws = [torch.empty(max(256, ops.prefix_workspace_bytes(9, 9, 1, 600, 384, 8, 2, 128, 16,
                                                          torch.bfloat16)),
                      dtype=torch.uint8, device=DEV) for _ in range(2)]

    def go(i):
        ops.paged_attention_decode_prefix(t["q"], t["kc"], t["vc"], table, bt, lens, pb["scale"],
                                          prefix_len=384, max_context_len=600, out=outs[i],
                                          workspace=ws[i])
    go(0)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, gr in enumerate(graphs):
        with torch.cuda.graph(gr):
            go(i)
    for it in range(3):
        t["q"].copy_(torch.randn(t["q"].shape).to(torch.bfloat16))
        lens.sub_(it)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        now = dict(pb, q=t["q"].cpu(), lens=lens.cpu().tolist())
        check(ops, now, outs[0])
        assert torch.equal(outs[0], outs[1])


def test_refused_arguments(ops):
    pb = problem([100, 120], [1, 1], 4, 2, 128, 16, 64, seed=2)
    with pytest.raises(ops.PagedKVError):
        call(ops, dict(pb, prefix=60))                          # not whole blocks
    with pytest.raises(ValueError):
        call(ops, dict(pb, prefix=96))                          # more than the table lists
    with pytest.raises(ops.PagedKVError):
        call(ops, dict(pb, scale=-1.0))
    with pytest.raises(ops.PagedKVError):
        call(ops, dict(pb, q=pb["q"].float(), kc=pb["kc"].float(), vc=pb["vc"].float()))
    with pytest.raises(TypeError):
        call(ops, dict(pb, q=pb["q"].float()))
    wide = problem([100, 120], [8, 8], 4, 2, 128, 16, 64, seed=2)
    with pytest.raises(ops.PagedKVError):
        call(ops, wide)                                         # 16 query rows per KV head
