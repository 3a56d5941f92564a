"""The operators of one step of a serving engine over the paged KV cache, as cases to measure.

A step with drafted tokens runs four of them, one after the other:

  tables   block tables, positions and token slots of the step's new tokens from the requests' lengths
  rope     RMS norms of the query and key heads, the rotation by position, and the write of K and V into the pages
  prefix   attention of the new tokens of a batch whose requests share a long prefix, the prefix read once for all
  verify   the drafted tokens against the target's probabilities, from given random numbers

`own` chooses between elementary torch operations (False) and the framework's calls (True).
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: a handful of block boundaries crossed, latency only
        dict(name="tables decode", op="tables", seqs=64, block=16, len_lo=512, len_hi=4096, new_lo=1, new_hi=1, over=0.0, shared=0),
        # admission of a few hundred prompts of very different lengths, a few requests over, a shared prefix that stays
        dict(name="tables prompts", op="tables", seqs=509, block=16, len_lo=128, len_hi=2048, new_lo=1, new_hi=4096, over=0.1, shared=8),
        # one decode step, query and key norms, grouped heads, rows cut out of one projection's output
        dict(name="rope decode", op="rope", tokens=64, heads=16, kv=8, dim=128, block=16, rot=128, norm=True, pairs=False, pool="bf16"),
        # a long chunk of prompts on a model without head norms
        dict(name="rope prompts", op="rope", tokens=16381, heads=32, kv=8, dim=128, block=16, rot=128, norm=False, pairs=False, pool="bf16"),
        # drafted tokens of a large batch into one-byte pages
        dict(name="rope fp8 pages", op="rope", tokens=1021, heads=64, kv=8, dim=128, block=32, rot=128, norm=True, pairs=False, pool="fp8"),
        # a few requests behind a short system prompt: latency
        dict(name="prefix small", op="prefix", seqs=4, rows=1, heads=16, kv=8, dim=128, block=16, prefix=512, tail_lo=1, tail_hi=100),
        # drafted tokens behind a prompt of a few thousand tokens
        dict(name="prefix drafts", op="prefix", seqs=61, rows=4, heads=16, kv=8, dim=128, block=16, prefix=4112, tail_lo=4, tail_hi=700),
        # a few requests over one very long document
        dict(name="prefix document", op="prefix", seqs=8, rows=1, heads=64, kv=8, dim=128, block=32, prefix=131072, tail_lo=16, tail_hi=2048),
        # many requests over one prompt, each with a part of its own: tensor work and page traffic at once
        dict(name="prefix many", op="prefix", seqs=1024, rows=1, heads=32, kv=8, dim=128, block=16, prefix=2048, tail_lo=16, tail_hi=1024),
        # one user, four drafted tokens: latency
        dict(name="verify one", op="verify", seqs=1, drafts=4, vocab=32000, dtype="float32"),
        # an ordinary batch, an odd vocabulary, 16-bit probabilities
        dict(name="verify odd", op="verify", seqs=61, drafts=3, vocab=50021, dtype="bfloat16"),
        # a large batch with a large vocabulary
        dict(name="verify large", op="verify", seqs=256, drafts=4, vocab=131072, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "prefix", "verify"])
    if op == "tables":
        lo = _log(rng, 1, 2048)
        return dict(op=op, seqs=_log(rng, 1, 509), block=rng.choice([8, 16, 32, 64]), len_lo=lo, len_hi=lo + _log(rng, 1, 2048), new_lo=rng.choice([0, 1]),
                    new_hi=_log(rng, 1, 4096), over=rng.choice([0.0, 0.1, 0.3]), shared=rng.choice([0, 1, 8]))
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128])
        return dict(op=op, tokens=_log(rng, 1, 8191), heads=kv * rng.choice([1, 2, 4, 7, 8]), kv=kv, dim=dim, block=rng.choice([8, 16, 32]),
                    rot=rng.choice([dim, dim, dim // 2]), norm=rng.choice([True, False]), pairs=rng.choice([False, False, True]), pool=rng.choice(["bf16", "bf16", "fp8", "f32"]))
    if op == "prefix":
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7, 8])
        rows = rng.choice([r for r in (1, 1, 2, 3, 4) if r * group <= 8])
        block = rng.choice([8, 16, 32])
        seqs = _log(rng, 1, 600)
        tail = _log(rng, 4, 1024)
        return dict(op=op, seqs=seqs, rows=rows, heads=kv * group, kv=kv, dim=rng.choice([64, 128, 128]), block=block, prefix=block * _log(rng, 1, min(4096, 131072 // block, 1200000 // (seqs * rows * group) + 1)),
                    tail_lo=rng.randint(rows, 2 * rows), tail_hi=tail + 2 * rows)
    return dict(op=op, seqs=_log(rng, 1, 200), drafts=rng.randint(0, 6), vocab=_log(rng, 1000, 131072), dtype=rng.choice(["float32", "float32", "bfloat16"]))


# ---------------------------------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"tables": _prepare_tables, "rope": _prepare_rope, "prefix": _prepare_prefix, "verify": _prepare_verify}[case["op"]](case, gen)
    st["case"] = case
    return st


def _ints(gen, lo, hi, shape, dtype=torch.int32):
    return torch.randint(int(lo), int(hi) + 1, shape, generator=gen, device=DEV, dtype=dtype)


def _page_rows(gen, blocks):
    """For each request as many pages as it needs, drawn without order from one pool: (table rows, pages in the pool, order of the free ones)."""
    need = int(blocks.sum())
    pool = need + need // 4 + 4
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    S, most = blocks.shape[0], int(blocks.max()) + 1
    at = torch.arange(most, device=DEV)[None]
    first = (torch.cumsum(blocks, 0) - blocks)[:, None]
    rows = torch.where(at < blocks[:, None], order[(first + at).clamp(max=pool - 1)], torch.zeros((), dtype=torch.int32, device=DEV))
    return rows.contiguous(), pool, order[need:]


def _token_bound(case):
    """Tokens that a step of these requests never exceeds: all of them at their most, or their mean and six deviations of the sum."""
    S, lo, hi = case["seqs"], case["new_lo"], case["new_hi"]
    return min(S * hi, int(S * (lo + hi) / 2 + 6 * math.sqrt(S / 12) * (hi - lo + 1)) + 1)


def _prepare_tables(case, gen):
    S, K = case["seqs"], case["block"]
    lens = _ints(gen, case["len_lo"], case["len_hi"], (S,)) + case["shared"] * K
    counts = _ints(gen, case["new_lo"], case["new_hi"], (S,))
    counts = torch.where(torch.rand(S, generator=gen, device=DEV) < case["over"], torch.full_like(counts, -1), counts)
    held = (lens + K - 1) // K
    width = (int(case["len_hi"]) + case["shared"] * K + int(case["new_hi"])) // K + 2
    blocks = S * width
    ring = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)[None]
    first = (torch.cumsum(held, 0) - held)[:, None]
    rows = torch.where(at < held[:, None], ring[(first + at).clamp(max=blocks - 1)], torch.full((), -7, dtype=torch.int32, device=DEV)).contiguous()
    state = torch.tensor([int(held.sum()), blocks], dtype=torch.int64, device=DEV)
    shared = torch.full((S,), case["shared"], dtype=torch.int32, device=DEV)
    cap = _token_bound(case)
    st = dict(lens=lens, counts=counts, held=held, rows=rows, ring=ring, state=state, shared=shared, blocks=blocks, cap=cap)
    st["outs"] = dict(context_lens=torch.empty_like(lens), cu_seqlens=torch.empty(S + 1, dtype=torch.int32, device=DEV),
                      cu_blocks=torch.empty(S + 1, dtype=torch.int32, device=DEV), positions=torch.empty(cap, dtype=torch.int32, device=DEV), slots=torch.empty(cap, dtype=torch.int64, device=DEV),
                      held_out=torch.empty_like(held), ring_state_out=torch.empty_like(state),
                      totals=torch.empty(4, dtype=torch.int32, device=DEV))
    return st


def _prepare_rope(case, gen):
    T, H, J, D, K = case["tokens"], case["heads"], case["kv"], case["dim"], case["block"]
    dt = torch.float32 if case["pool"] == "f32" else torch.bfloat16
    qkv = torch.randn((T, (H + 2 * J) * D), generator=gen, device=DEV).to(dt)
    blocks = -(-T // K) * 5 // 4 + 2
    slots = torch.randperm(blocks * K, generator=gen, device=DEV)[:T].contiguous()
    far = 32768
    positions = _ints(gen, 0, far - 1, (T,))
    rot = case["rot"]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * inv[None]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    st = dict(q=qkv[:, :H * D].view(T, H, D), k=qkv[:, H * D:(H + J) * D].view(T, J, D), v=qkv[:, (H + J) * D:].view(T, J, D),
              slots=slots, positions=positions, cos_sin=cos_sin, eps=1e-6)
    st["wq"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) if case["norm"] else None
    st["wk"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) if case["norm"] else None
    if case["pool"] == "fp8":
        st["kc"] = torch.zeros((blocks, K, J, D), dtype=torch.uint8, device=DEV)
        st["vc"] = torch.zeros((blocks, K, J, D), dtype=torch.uint8, device=DEV)
    else:
        st["kc"] = torch.zeros((blocks, K, J, D), dtype=dt, device=DEV)
        st["vc"] = torch.zeros((blocks, K, J, D), dtype=dt, device=DEV)
    st["q_out"] = torch.empty((T, H, D), dtype=dt, device=DEV)
    if own:
        from paged_kv_cache_115_gb300 import ops
        st["quant"] = ops.kv_quant("fp8", 0.03125, 0.015625) if case["pool"] == "fp8" else None
    return st


def _prepare_prefix(case, gen):
    S, N, H, J, D, K, P = (case[k] for k in ("seqs", "rows", "heads", "kv", "dim", "block", "prefix"))
    tail = _ints(gen, case["tail_lo"], case["tail_hi"], (S,))
    shared = P // K
    own_rows, pool, _ = _page_rows(gen, (tail + K - 1) // K)
    pool += shared
    table = (torch.arange(shared, device=DEV) * 7919 % shared).to(torch.int32) if shared % 7919 else torch.arange(shared, device=DEV, dtype=torch.int32)
    rows = torch.cat([table[None].expand(S, -1), own_rows + shared], 1).contiguous()
    kc = torch.empty((pool, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    vc = torch.empty((pool, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    if N > 1:  # drafted tokens: one to `rows` of them a request, packed
        n = (torch.arange(S, device=DEV, dtype=torch.int32) * 5 % N) + 1
    else:
        n = torch.ones(S, dtype=torch.int32, device=DEV)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), torch.cumsum(n, 0).to(torch.int32)])
    T = int(cu[-1])
    q = torch.randn((T, H, D), generator=gen, device=DEV).to(torch.bfloat16)
    st = dict(q=q, kc=kc, vc=vc, table=table.contiguous(), rows=rows, lens=(tail + P).to(torch.int32), cu=cu, scale=D ** -0.5,
              most=P + case["tail_hi"], out=torch.empty_like(q))
    if own:
        from paged_kv_cache_115_gb300 import ops
        need = ops.prefix_workspace_bytes(S, T, N, st["most"], P, H, J, D, K, torch.bfloat16)
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


def _prepare_verify(case, gen):
    S, N, V = case["seqs"], case["drafts"], case["vocab"]
    dt = getattr(torch, case["dtype"])
    n = _ints(gen, max(0, N - 1), N, (S,)) if S > 1 else torch.full((S,), N, dtype=torch.int32, device=DEV)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), torch.cumsum(n + 1, 0).to(torch.int32)])
    T = int(cu[-1])
    logits = torch.randn((T, V), generator=gen, device=DEV) * 3
    target = torch.softmax(logits, -1).to(dt)
    tokens = torch.zeros(T, dtype=torch.int32, device=DEV)
    draft = torch.zeros((S, max(N, 1), V), dtype=dt, device=DEV)
    s = torch.repeat_interleave(torch.arange(S, device=DEV), (n + 1).long(), output_size=T)
    i = torch.arange(T, device=DEV) - cu[s]
    rows = torch.nonzero(i < n[s])[:, 0]
    if rows.numel():
        q = torch.softmax(logits[rows] + 0.7 * torch.randn((rows.numel(), V), generator=gen, device=DEV), -1)
        tokens[rows + 1] = torch.multinomial(q, 1, generator=gen)[:, 0].to(torch.int32)
        draft[s[rows], i[rows]] = q.to(dt)
    uniforms = torch.rand(T, generator=gen, device=DEV)
    return dict(target=target, draft=draft if N else None, tokens=tokens, uniforms=uniforms, cu=cu, most=N + 1,
                out=torch.empty((S, N + 1), dtype=torch.int32, device=DEV), new=torch.empty(S, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "prefix": _own_prefix, "verify": _own_verify}[st["case"]["op"]](st)
    return {"tables": _plain_tables, "rope": _plain_rope, "prefix": _plain_prefix, "verify": _plain_verify}[st["case"]["op"]](st)


def _own_tables(st):
    from paged_kv_cache_115_gb300 import ops
    o = st["outs"]
    ops.step_tables(st["lens"], st["counts"], st["rows"], st["held"], st["ring"], st["state"], st["case"]["block"], st["blocks"],
                    shared=st["shared"], **o)
    return {"rows": st["rows"], "ring": st["ring"], **o}


def _own_rope(st):
    from paged_kv_cache_115_gb300 import ops
    ops.paged_qk_norm_rope_append(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["kc"], st["vc"], st["cos_sin"],
                                  q_weight=st["wq"], k_weight=st["wk"], eps=st["eps"], interleaved=st["case"]["pairs"],
                                  quant=st["quant"], q_out=st["q_out"])
    return _rope_outputs(st)


def _own_prefix(st):
    from paged_kv_cache_115_gb300 import ops
    cu = st["cu"] if st["case"]["rows"] > 1 else None
    ops.paged_attention_decode_prefix(st["q"], st["kc"], st["vc"], st["table"], st["rows"], st["lens"], st["scale"],
                                      prefix_len=st["case"]["prefix"], max_context_len=st["most"], cu_seqlens=cu,
                                      max_query_len=st["case"]["rows"], out=st["out"], workspace=st["ws"])
    return st["out"]


def _own_verify(st):
    from paged_kv_cache_115_gb300 import ops
    ops.verify_draft_tokens(st["target"], st["draft"], st["tokens"], st["uniforms"], st["cu"], st["most"],
                            out_tokens=st["out"], num_new=st["new"])
    return {"tokens": st["out"], "new": st["new"]}


def _plain_tables(st):
    K, rows, ring = st["case"]["block"], st["rows"], st["ring"]
    lens, held, shared = st["lens"].long(), st["held"].long(), st["shared"].long()
    over = st["counts"] < 0
    n = st["counts"].long().clamp(min=0)
    ctx = torch.where(over, 0, lens + n)
    need = (ctx + K - 1) // K
    take = torch.where(over, 0, (need - held).clamp(min=0))
    give = torch.where(over, (held - shared).clamp(min=0), 0)
    cu = torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])
    size = ring.shape[0]
    at = torch.arange(rows.shape[1], device=rows.device)[None]
    # pages of the finished requests go behind the ring's end, those taken come from its start
    back = over[:, None] & (at >= shared[:, None]) & (at < held[:, None])
    where = (st["state"][1] + (torch.cumsum(give, 0) - give)[:, None] + at - shared[:, None]) % size
    longer = torch.cat([ring, ring[:1]])
    longer[torch.where(back, where, size)] = rows
    fresh = ~over[:, None] & (at >= held[:, None]) & (at < need[:, None])
    where = (st["state"][0] + (torch.cumsum(take, 0) - take)[:, None] + at - held[:, None]) % size
    rows.copy_(torch.where(fresh, ring[where], rows))
    ring.copy_(longer[:size])
    t = torch.arange(st["cap"], device=rows.device)
    s = torch.searchsorted(cu[1:], t, right=True).clamp(max=n.shape[0] - 1)
    live = t < cu[-1]
    pos = torch.where(live, ctx[s] - n[s] + t - cu[s], -1)
    page = rows[s, (pos.clamp(min=0) // K)].long()
    slots = torch.where(live, page * K + pos % K, -1)
    total = torch.stack([torch.zeros_like(cu[-1]), cu[-1], take.sum(), give.sum()])
    return {"rows": rows, "ring": ring, "context_lens": ctx.int(), "cu_seqlens": cu.int(),
            "cu_blocks": torch.cat([torch.zeros_like(n[:1]), torch.cumsum(take, 0)]).int(), "positions": pos.int(), "slots": slots,
            "held_out": torch.where(over, 0, torch.maximum(held, need)).int(), "ring_state_out": st["state"] + torch.stack([take.sum(), give.sum()]),
            "totals": total.int()}


def _rope_outputs(st):
    kc, vc = st["kc"], st["vc"]
    if st["case"]["pool"] == "fp8":  # codes as the values they stand for
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    return {"q": st["q_out"], "k_cache": kc, "v_cache": vc}


def _normed(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _turned(x, cs, rot, pairs):
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(st):
    case, dt = st["case"], st["q"].dtype
    cs = st["cos_sin"][st["positions"].long()]
    st["q_out"].copy_(_turned(_normed(st["q"], st["wq"], st["eps"]), cs, case["rot"], case["pairs"]))
    k = _turned(_normed(st["k"], st["wk"], st["eps"]), cs, case["rot"], case["pairs"])
    J, D = case["kv"], case["dim"]
    if case["pool"] == "fp8":
        k = (k / 0.03125).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (st["v"].float() / 0.015625).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        k, v = k.to(dt), st["v"]
    st["kc"].view(-1, J, D)[st["slots"]] = k
    st["vc"].view(-1, J, D)[st["slots"]] = v
    return _rope_outputs(st)


def _plain_prefix(st):
    S, N, H, J, D, K, P = (st["case"][k] for k in ("seqs", "rows", "heads", "kv", "dim", "block", "prefix"))
    G, q, cu = H // J, st["q"], st["cu"].long()
    T = q.shape[0]
    kp = st["kc"][st["table"].long()].view(P, J, D).float().permute(1, 0, 2)
    vp = st["vc"][st["table"].long()].view(P, J, D).float().permute(1, 0, 2)
    qs = q.float().view(T, J, G, D).permute(1, 0, 2, 3).reshape(J, T * G, D)
    front = (torch.matmul(qs, kp.transpose(1, 2)) * st["scale"]).view(J, T, G, P)
    # each request's own tokens, padded to the longest
    pages = st["rows"][:, P // K:].long()
    L = pages.shape[1] * K
    kt = st["kc"][pages].view(S, L, J, D).permute(0, 2, 1, 3).float()
    vt = st["vc"][pages].view(S, L, J, D).permute(0, 2, 1, 3).float()
    n = cu[1:] - cu[:-1]
    i = torch.arange(N, device=q.device)
    at = (cu[:-1, None] + i[None]).clamp(max=T - 1)                       # packed row of request s's token i
    qt = q[at].view(S, N, J, G, D).permute(0, 2, 1, 3, 4).reshape(S, J, N * G, D).float()
    back = (torch.matmul(qt, kt.transpose(2, 3)) * st["scale"]).view(S, J, N, G, L)
    last = (st["lens"].long() - P)[:, None] - n[:, None] + i[None]        # last own token that row i sees
    back = torch.where(torch.arange(L, device=q.device)[None, None] <= last[:, :, None], 0.0, -math.inf)[:, None, :, None] + back
    s = torch.searchsorted(cu[1:], torch.arange(T, device=q.device), right=True)
    r = torch.arange(T, device=q.device) - cu[s]
    back_t = back.permute(0, 2, 1, 3, 4)[s, r].permute(1, 0, 2, 3)        # [J, T, G, L]
    top = torch.maximum(front.amax(-1), back_t.amax(-1))
    front = torch.exp(front - top[..., None])
    full = torch.zeros((S, N, J, G), device=q.device)
    full[s, r] = top.permute(1, 0, 2)
    back = torch.exp(back - full.permute(0, 2, 1, 3)[..., None])
    o = torch.matmul(front.view(J, T * G, P), vp).view(J, T, G, D)
    ot = torch.matmul(back.reshape(S, J, N * G, L), vt).view(S, J, N, G, D)
    o = o + ot.permute(0, 2, 1, 3, 4)[s, r].permute(1, 0, 2, 3)
    total = front.sum(-1) + back.sum(-1).permute(0, 2, 1, 3)[s, r].permute(1, 0, 2)
    st["out"].copy_((o / total[..., None]).permute(1, 0, 2, 3).reshape(T, H, D))
    return st["out"]


def _plain_verify(st):
    target, draft, tokens, cu = st["target"], st["draft"], st["tokens"].long(), st["cu"].long()
    S, V = cu.shape[0] - 1, target.shape[1]
    n = cu[1:] - cu[:-1] - 1
    sid = torch.arange(S, device=target.device)
    if draft is not None:
        i = torch.arange(draft.shape[1], device=target.device)[None]
        live = i < n[:, None]
        row = torch.where(live, cu[:-1, None] + i, 0)
        token = torch.where(live, tokens[(row + 1).clamp(max=tokens.shape[0] - 1)], 0)
        p = target[row, token].double()
        q = draft[sid[:, None], i, token].double()
        good = live & (st["uniforms"][row].double() * q < p)
        a = torch.cumprod(good.long(), 1).sum(1)
    else:
        a = torch.zeros_like(n)
    w = target[cu[:-1] + a].float()
    p = w
    if draft is not None:
        refused = (a < n)[:, None]
        w = torch.where(refused, w - draft[sid, torch.minimum(a, n - 1).clamp(min=0)].float(), w)
    parts = (w.clamp(0, 1).double() * 2.0 ** 40).long()
    total = parts.sum(1, keepdim=True)
    parts = torch.where(total == 0, (p.clamp(0, 1).double() * 2.0 ** 40).long(), parts)
    sums = torch.cumsum(parts, 1)
    total = sums[:, -1]
    u = (st["uniforms"][cu[1:] - 1].double() * 2.0 ** 24).long()
    r = (total >> 24) * u + (((total & 0xFFFFFF) * u) >> 24)
    new = (sums <= r[:, None]).sum(1)
    i = torch.arange(st["most"], device=target.device)[None]
    taken = tokens[(cu[:-1, None] + 1 + i).clamp(max=tokens.shape[0] - 1)]
    out = torch.where(i < a[:, None], taken, torch.where(i == a[:, None], new[:, None], -1))
    return {"tokens": out.int(), "new": (a + 1).int()}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "tables":
        S, K = case["seqs"], case["block"]
        over = case["over"]
        tokens = S * (1 - over) * (case["new_lo"] + case["new_hi"]) / 2
        pages = tokens / K + S * over * (case["len_lo"] + case["len_hi"]) / 2 / K
        return {"bytes": S * 4 * 8 + pages * 8 + _token_bound(case) * 12, "flops": 0}
    if case["op"] == "rope":
        T, H, J, D = case["tokens"], case["heads"], case["kv"], case["dim"]
        e = 4 if case["pool"] == "f32" else 2
        o = 1 if case["pool"] == "fp8" else e
        return {"bytes": T * ((2 * H + 2 * J) * D * e + 2 * J * D * o + 4 * case["rot"] + 12), "flops": T * (H + J) * D * (7 if case["norm"] else 3)}
    if case["op"] == "prefix":
        S, N, H, J, D, P = (case[k] for k in ("seqs", "rows", "heads", "kv", "dim", "prefix"))
        tail = (case["tail_lo"] + case["tail_hi"]) / 2
        rows = S * (N + 1) / 2
        return {"bytes": (P + S * tail) * J * D * 4 + rows * H * D * 4, "flops": 4 * rows * H * D * (P + tail)}
    S, N, V = case["seqs"], case["drafts"], case["vocab"]
    e = 4 if case["dtype"] == "float32" else 2
    # the target's row of the first refused token (or the last one), and the draft's where one was refused (about three in four requests)
    return {"bytes": S * V * e * (1.75 if N else 1) + S * (N + 1) * 16, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits (whole numbers have none of their own)
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("tables", "verify"):
        return None
    st = prepare(case, seed)
    return _exact_rope(case, st) if case["op"] == "rope" else _exact_prefix(case, st)


def _exact_rope(case, st):
    D, half, pos = case["dim"], case["rot"] // 2, st["positions"].long()

    def through(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(torch.sum(y ** 2, 2, True) / D + st["eps"]) * w.double()
        # each rotated pair as a complex number
        table = st["cos_sin"][pos].double()
        unit = torch.complex(table[:, :half], table[:, half:]).unsqueeze(1)
        j = torch.arange(half, device=x.device)
        lo, hi = (2 * j, 2 * j + 1) if case["pairs"] else (j, j + half)
        z = torch.complex(y[:, :, lo], y[:, :, hi]) * unit
        y[:, :, lo], y[:, :, hi] = z.real, z.imag
        return y

    ks, vs = (0.03125, 0.015625) if case["pool"] == "fp8" else (1.0, 1.0)
    kc = torch.zeros(st["kc"].shape, dtype=torch.float64, device=DEV)
    vc = torch.zeros_like(kc)
    kc.flatten(0, 1)[st["slots"]] = through(st["k"], st["wk"]) / ks
    vc.flatten(0, 1)[st["slots"]] = st["v"].double() / vs
    if case["pool"] == "fp8":
        kc, vc = kc.clamp(-448, 448), vc.clamp(-448, 448)
    return {"q": through(st["q"], st["wq"]), "k_cache": kc, "v_cache": vc}


def _exact_prefix(case, st):
    S, H, J, D, K = (case[k] for k in ("seqs", "heads", "kv", "dim", "block"))
    G = H // J
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    for s in range(S):
        n, L = cu[s + 1] - cu[s], lens[s]
        t = torch.arange(L, device=DEV)
        slot = st["rows"][s].long()[t // K] * K + t % K
        k = st["kc"].flatten(0, 1)[slot].double().permute(1, 2, 0)         # [J, D, L]
        v = st["vc"].flatten(0, 1)[slot].double().permute(1, 0, 2)         # [J, L, D]
        q = st["q"][cu[s]:cu[s + 1]].double().view(n, J, G, D).permute(1, 0, 2, 3).reshape(J, n * G, D)
        x = (q @ k) * st["scale"]
        last = torch.arange(L - n, L, device=DEV).repeat_interleave(G)
        x = x.masked_fill(t[None, None, :] > last[None, :, None], -math.inf)
        o = torch.softmax(x, -1) @ v
        out[cu[s]:cu[s + 1]] = o.view(J, n, G, D).permute(1, 0, 2, 3).reshape(n, H, D)
    return out
