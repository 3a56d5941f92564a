"""Operators of beam search over a paged KV cache held in 4 bits, as cases to measure.

A step of beam search runs them one after the other, the attention and the writes once per layer:

  write    the new tokens' K and V rows into 4-bit pages, one scale and one offset per token and KV head
  attn     decode attention over 4-bit pages; beams of one request list the same pages for what they share
  select   the best candidates over a request's beams and the vocabulary, from logits and the beams' scores
  fork     the chosen beams' block tables: shared pages, fresh ones for partly filled pages and their copy, free pages back

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
        # one decode step of a batch of requests: a row each, latency
        dict(name="write decode", op="write", tokens=64, kv=8, dim=128, block=16, dtype="bfloat16"),
        # the prompts of a batch, K and V cut out of one projection's output
        dict(name="write prompts", op="write", tokens=16381, kv=8, dim=128, block=16, dtype="bfloat16"),
        # a few requests with short histories: latency
        dict(name="attn small", op="attn", seqs=4, group=1, heads=16, kv=8, dim=128, block=16, len_lo=100, len_hi=512, own_hi=0, share=False),
        # an ordinary batch of ragged lengths
        dict(name="attn batch", op="attn", seqs=61, group=1, heads=16, kv=8, dim=128, block=16, len_lo=1, len_hi=4096, own_hi=0, share=False),
        # a large batch with long histories
        dict(name="attn large", op="attn", seqs=128, group=1, heads=32, kv=8, dim=128, block=16, len_lo=1024, len_hi=8192, own_hi=0, share=False),
        # a few very long documents, many query heads to a KV head
        dict(name="attn document", op="attn", seqs=4, group=1, heads=64, kv=8, dim=128, block=32, len_lo=131072, len_hi=131072, own_hi=0, share=False),
        # beam search: 48 requests of 4 beams that share a prompt and part ways in their last tokens
        dict(name="attn beams", op="attn", seqs=192, group=4, heads=32, kv=8, dim=128, block=16, len_lo=1024, len_hi=4096, own_hi=300, share=True),
        # one request, four beams: latency
        dict(name="select one", op="select", requests=1, beams=4, vocab=32000, take=4, over=0.0, dtype="float32"),
        # an ordinary batch, twice as many candidates as beams, an odd vocabulary, some beams at their end
        dict(name="select odd", op="select", requests=13, beams=5, vocab=50021, take=10, over=0.2, dtype="bfloat16"),
        # a large batch with a large vocabulary
        dict(name="select large", op="select", requests=64, beams=8, vocab=131072, take=8, over=0.05, dtype="bfloat16"),
        # a few requests in one layer's 4-bit pages: latency
        dict(name="fork small", op="fork", requests=8, beams=4, block=16, len_lo=64, len_hi=512, own_hi=64, over=0.1, layers=1, kv=8, dim=128, pool="int4"),
        # a large batch, the bf16 pages of two layers
        dict(name="fork large", op="fork", requests=61, beams=8, block=16, len_lo=512, len_hi=2048, own_hi=300, over=0.1, layers=2, kv=8, dim=128, pool="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attn", "attn", "select", "fork"])
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 8191), kv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 128]), block=rng.choice([8, 16, 32]),
                    dtype=rng.choice(["bfloat16", "bfloat16", "float32"]))
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 1, 2, 4, 5, 8])
        hi = _log(rng, 1, 32768)
        most = max(1, min(512, 700000 // (hi + 300)) // group)
        return dict(op=op, seqs=group * _log(rng, 1, most), group=group, heads=kv * rng.choice([1, 2, 4, 7, 8]), kv=kv, dim=128, block=rng.choice([8, 16, 32, 64]),
                    len_lo=rng.randint(0 if group == 1 else 1, hi), len_hi=hi, own_hi=_log(rng, 1, 300) if group > 1 else 0, share=group > 1)
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _log(rng, 1000, 131072)
        return dict(op=op, requests=_log(rng, 1, max(1, min(128, 60000000 // (beams * vocab)))), beams=beams, vocab=vocab,
                    take=rng.choice([max(beams, 2), min(32, 2 * beams)]), over=rng.choice([0.0, 0.0, 0.2]), dtype=rng.choice(["bfloat16", "float32"]))
    beams = rng.choice([2, 3, 4, 5, 8])
    lo = _log(rng, 1, 2048)
    return dict(op=op, requests=_log(rng, 1, 48), beams=beams, block=rng.choice([8, 16, 32]), len_lo=lo, len_hi=lo + _log(rng, 1, 2048), own_hi=_log(rng, 2, 300),
                over=rng.choice([0.0, 0.1, 0.5]), layers=rng.choice([1, 1, 2]), kv=rng.choice([1, 2, 4, 8]), dim=128, pool=rng.choice(["bf16", "int4"]))


# ---------------------------------------------------------------------------------------------------------------------
# 4-bit rows: per token and KV head x ~ offset + scale * code, code 0 .. 15, element 2 i in the low half of byte i
# ---------------------------------------------------------------------------------------------------------------------

def _down(x):
    """float32 to the next bfloat16 at or below it."""
    bits = x.contiguous().view(torch.int32)
    cut = bits & -65536
    cut = torch.where((bits < 0) & (bits != cut), cut + 65536, cut)
    return cut.view(torch.float32).to(torch.bfloat16)


def _quantize(x):
    """[..., D] -> (codes uint8 [..., D / 2], bfloat16 [..., 2]: scale and offset; a pool keeps these as [pages, heads, tokens, 2])."""
    x = x.float()
    offset = _down(x.amin(-1))
    scale = ((x.amax(-1) - offset.float()) / 15).to(torch.bfloat16)
    inv = torch.where(scale.float() >= 2.0 ** -126, 1 / scale.float(), 0)
    codes = ((x - offset.float()[..., None]) * inv[..., None]).round().clamp(0, 15).to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), torch.stack([scale, offset], -1)


def _values(codes, scales):
    """What 4-bit rows stand for, float32."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return c * scales[..., 0, None].float() + scales[..., 1, None].float()


def _pool4(gen, blocks, K, J, D):
    """A pool of normal rows held in 4 bits: (codes, scales)."""
    codes = torch.empty((blocks, K, J, D // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((blocks, J, K, 2), dtype=torch.bfloat16, device=DEV)
    part = max(1, (1 << 26) // (K * J * D))
    for b in range(0, blocks, part):
        n = min(part, blocks - b)
        c, s = _quantize(torch.randn((n, K, J, D), generator=gen, device=DEV))
        codes[b:b + n], scales[b:b + n] = c, s.transpose(1, 2)
    return codes, scales


# ---------------------------------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"write": _prepare_write, "attn": _prepare_attn, "select": _prepare_select, "fork": _prepare_fork}[case["op"]](case, gen)
    st["case"] = case
    return st


def _ints(gen, lo, hi, shape, dtype=torch.int32):
    return torch.randint(int(lo), int(hi) + 1, shape, generator=gen, device=DEV, dtype=dtype)


def _quant4(ks, vs):
    from paged_kv_cache_115_gb300 import ops
    return ops.kv_quant("int4", k_token_scales=ks, v_token_scales=vs)


def _prepare_write(case, gen):
    T, J, D, K = case["tokens"], case["kv"], case["dim"], case["block"]
    dt = getattr(torch, case["dtype"])
    # K rows and V rows as the projection leaves them, its channels of different sizes
    width = torch.rand(2 * J * D, generator=gen, device=DEV) * 2 + 0.25
    kv = (torch.randn((T, 2 * J * D), generator=gen, device=DEV) * width).to(dt)
    blocks = -(-T // K) * 5 // 4 + 2
    slots = torch.randperm(blocks * K, generator=gen, device=DEV)[:T].contiguous()
    st = dict(k=kv[:, :J * D].view(T, J, D), v=kv[:, J * D:].view(T, J, D), slots=slots)
    for n in ("k", "v"):
        st[n + "c"] = torch.zeros((blocks, K, J, D // 2), dtype=torch.uint8, device=DEV)
        st[n + "s"] = torch.zeros((blocks, J, K, 2), dtype=torch.bfloat16, device=DEV)
    if own:
        st["quant"] = _quant4(st["ks"], st["vs"])
    return st


def _beam_rows(gen, lens, own_len, group, K, len_hi, own_hi):
    """Block tables of groups of rows that list the same pages for what they share: rows of a group share their first
    lens - own_len tokens' whole pages, and each has pages of its own behind.  Returns (rows, pages of the pool, the free ones
    among them in a buffer of fixed size and their number, listed entries)."""
    S = lens.shape[0]
    common = (lens - own_len).clamp(min=0) // K                                    # shared whole pages
    common = common.view(-1, group).amin(1, True).expand(-1, group).reshape(S) if group > 1 else torch.zeros_like(lens)
    held = (lens + K - 1) // K
    leader = torch.arange(S, device=DEV) // group * group
    first = torch.arange(S, device=DEV) == leader
    mine = held - torch.where(first, 0, common)                                    # pages that this row adds
    need = mine.sum()
    # room for every draw of the lengths, and a quarter more
    pool = S // group * (-(-len_hi // K) + group * (-(-own_hi // K) + 2)) * 5 // 4 + 4
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    start = torch.cumsum(mine, 0) - mine
    at = torch.arange(-(-(len_hi + own_hi) // K) + 1, device=DEV)[None]
    at_own = start[:, None] + at - torch.where(first, 0, common)[:, None]
    at_lead = start[leader][:, None] + at
    where = torch.where(at < common[:, None], at_lead, at_own).clamp(0, pool - 1)
    rows = torch.where(at < held[:, None], order[where], torch.full((), -7, dtype=torch.int32, device=DEV))
    free = order.roll(-int(need))
    return rows.contiguous(), pool, free, pool - int(need), held


def _prepare_attn(case, gen):
    S, g, H, J, D, K = (case[k] for k in ("seqs", "group", "heads", "kv", "dim", "block"))
    lens = _ints(gen, case["len_lo"], case["len_hi"], (S // g,), torch.int64).repeat_interleave(g)
    own_len = _ints(gen, 1, case["own_hi"], (S // g,), torch.int64).repeat_interleave(g) if g > 1 else torch.zeros_like(lens)
    lens = lens + own_len
    rows, pool, _, _, _ = _beam_rows(gen, lens, own_len, g, K, case["len_hi"], case["own_hi"])
    kc, ks = _pool4(gen, pool, K, J, D)
    vc, vs = _pool4(gen, pool, K, J, D)
    q = torch.randn((S, H, D), generator=gen, device=DEV).to(torch.bfloat16)
    st = dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, rows=rows, lens=lens.to(torch.int32), scale=D ** -0.5, most=case["len_hi"] + case["own_hi"], out=torch.empty_like(q))
    if own:
        from paged_kv_cache_115_gb300 import ops
        st["quant"] = _quant4(ks, vs)
        need = ops.attention_quant_workspace_bytes(S, H, J, D, K, st["most"], torch.bfloat16, st["quant"], share_prefix=case["share"])
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


def _prepare_select(case, gen):
    R, B, V, N = (case[k] for k in ("requests", "beams", "vocab", "take"))
    logits = (torch.randn((R * B, V), generator=gen, device=DEV) * 3).to(getattr(torch, case["dtype"]))
    scores = -5 - 4 * torch.rand((R, B), generator=gen, device=DEV)
    over = torch.rand((R, B), generator=gen, device=DEV) < case["over"]
    st = dict(logits=logits, scores=scores, over=over, eos=2,
              tokens=torch.empty((R, N), dtype=torch.int32, device=DEV), parents=torch.empty((R, N), dtype=torch.int32, device=DEV),
              scores_out=torch.empty((R, N), dtype=torch.float32, device=DEV), over_out=torch.empty((R, N), dtype=torch.bool, device=DEV))
    if own:
        from paged_kv_cache_115_gb300 import ops
        need = ops.beam_select_workspace_bytes(R, B, V, N)
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


def _prepare_fork(case, gen):
    R, B, K, L, J, D = (case[k] for k in ("requests", "beams", "block", "layers", "kv", "dim"))
    S = R * B
    lens = _ints(gen, case["len_lo"], case["len_hi"], (R,), torch.int64).repeat_interleave(B)
    own_len = _ints(gen, 1, case["own_hi"], (R,), torch.int64).repeat_interleave(B)
    lens = lens + own_len
    rows, pool, ring, free, held = _beam_rows(gen, lens, own_len, B, K, case["len_hi"], case["own_hi"])
    # the beams that the selection keeps; whole requests that are over
    parents = _ints(gen, 0, B - 1, (R, B))
    parents[torch.rand(R, generator=gen, device=DEV) < case["over"]] = -1
    st = dict(rows=rows, lens=lens.to(torch.int32), held=held.to(torch.int32), parents=parents, ring=ring.contiguous(), blocks=pool,
              state=torch.tensor([0, free], dtype=torch.int64, device=DEV))
    if case["pool"] == "int4":
        for n in ("k", "v"):
            st[n + "c"] = _ints(gen, 0, 255, (L, pool, K, J, D // 2), torch.uint8)
            st[n + "s"] = torch.rand((L, pool, J, K, 2), generator=gen, device=DEV).to(torch.bfloat16)
    else:
        for n in ("k", "v"):
            st[n + "c"] = torch.empty((L, pool, K, J, D), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    st["outs"] = dict(block_tables_out=torch.full_like(rows, -7), lens_out=torch.empty_like(st["lens"]), held_out=torch.empty_like(st["held"]),
                      ring_state_out=torch.empty_like(st["state"]), pairs=torch.empty((S, 2), dtype=torch.int64, device=DEV), totals=torch.empty(4, dtype=torch.int32, device=DEV))
    if own:
        from paged_kv_cache_115_gb300 import ops
        st["quant"] = _quant4(st["ks"], st["vs"]) if case["pool"] == "int4" else None
        need = ops.fork_workspace_bytes(R, B, rows.shape[1])
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return {"write": _own_write, "attn": _own_attn, "select": _own_select, "fork": _own_fork}[st["case"]["op"]](st)
    return {"write": _plain_write, "attn": _plain_attn, "select": _plain_select, "fork": _plain_fork}[st["case"]["op"]](st)


def _own_write(st):
    from paged_kv_cache_115_gb300 import ops
    ops.paged_kv_write_quant(st["k"], st["v"], st["slots"], st["kc"], st["vc"], st["quant"])
    return _write_outputs(st)


def _own_attn(st):
    from paged_kv_cache_115_gb300 import ops
    ops.paged_attention_decode_quant(st["q"], st["kc"], st["vc"], st["rows"], st["lens"], st["scale"], st["quant"], out=st["out"],
                                     max_context_len=st["most"], workspace=st["ws"], share_prefix=st["case"]["share"])
    return st["out"]


def _own_select(st):
    from paged_kv_cache_115_gb300 import ops
    ops.beam_select(st["logits"], st["scores"], st["case"]["take"], finished=st["over"], eos_token=st["eos"], tokens=st["tokens"],
                    parents=st["parents"], scores_out=st["scores_out"], finished_out=st["over_out"], workspace=st["ws"])
    return _select_outputs(st)


def _own_fork(st):
    from paged_kv_cache_115_gb300 import ops
    o = st["outs"]
    ops.fork_tables(st["parents"], st["lens"], st["held"], st["rows"], st["ring"], st["state"], st["case"]["block"], workspace=st["ws"], **o)
    ops.kv_fork_copy(st["kc"], st["vc"], o["pairs"], o["lens_out"], quant=st["quant"])
    return _fork_outputs(st)


def _write_outputs(st):
    """The pages: scales and offsets, and the codes, which float32 arithmetic fixes to the bit, as whole numbers (two to a byte)."""
    return {"k": st["kc"], "k_scales": st["ks"], "v": st["vc"], "v_scales": st["vs"]}


def _plain_write(st):
    K = st["case"]["block"]
    for n in ("k", "v"):
        codes, scales = _quantize(st[n])
        st[n + "c"].flatten(0, 1)[st["slots"]] = codes
        st[n + "s"][st["slots"] // K, :, st["slots"] % K] = scales
    return _write_outputs(st)


def _plain_attn(st):
    S, H, J, D, K = (st["case"][k] for k in ("seqs", "heads", "kv", "dim", "block"))
    G, q, lens = H // J, st["q"], st["lens"].long()
    width = st["rows"].shape[1]
    # eight sequences at a time, padded to the longest row
    for a in range(0, S, 8):
        b = min(S, a + 8)
        t = torch.arange(width * K, device=q.device)
        live = t[None] < lens[a:b, None]
        pages = st["rows"][a:b].long()
        pages = torch.where(torch.arange(width, device=q.device)[None] * K < lens[a:b, None], pages, 0)
        slot = (pages[:, :, None] * K + torch.arange(K, device=q.device)).flatten(1)
        k = _values(st["kc"].flatten(0, 1)[slot], st["ks"][slot // K, :, slot % K])  # [s, t, J, D]
        x = torch.matmul(q[a:b].view(b - a, J, G, D).float(), k.permute(0, 2, 3, 1)) * st["scale"]
        x = torch.where(live[:, None, None], x, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, 0, top))
        total = p.sum(-1, keepdim=True)
        del k, x
        v = _values(st["vc"].flatten(0, 1)[slot], st["vs"][slot // K, :, slot % K])
        o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1, total)
        st["out"][a:b] = o.view(b - a, H, D)
    return st["out"]


def _select_outputs(st):
    return {"tokens": st["tokens"], "parents": st["parents"], "scores": st["scores_out"], "finished": st["over_out"]}


def _plain_select(st):
    R, B, V, N = (st["case"][k] for k in ("requests", "beams", "vocab", "take"))
    x = st["logits"].double()                       # 64 bits: candidates of two beams may lie next to each other
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    x = (x - lse).view(R, B, V) + st["scores"].double()[..., None]
    ended = torch.full_like(x, -math.inf)
    ended[..., st["eos"]] = st["scores"].double()
    x = torch.where(st["over"][..., None], ended, x).flatten(1)
    at = torch.arange(B * V, device=x.device)[None]
    free = torch.ones_like(x, dtype=torch.bool)
    for n in range(N):
        best = torch.where(free, x, -math.inf).amax(1, keepdim=True)
        i = torch.where(free & (x == best), at, B * V).amin(1, keepdim=True)
        free.scatter_(1, i, False)
        none = best[:, 0] == -math.inf              # fewer candidates than asked for
        parent, token = torch.where(none, -1, i[:, 0] // V), torch.where(none, -1, i[:, 0] % V)
        st["parents"][:, n], st["tokens"][:, n], st["scores_out"][:, n] = parent, token, best[:, 0]
        st["over_out"][:, n] = none | st["over"].gather(1, parent.clamp(min=0)[:, None])[:, 0] | (token == st["eos"])
    return _select_outputs(st)


def _fork_outputs(st):
    o = dict(st["outs"])
    o["ring"] = st["ring"]
    o["k_cache"], o["v_cache"] = st["kc"], st["vc"]
    if st["case"]["pool"] == "int4":
        o["k_scales"], o["v_scales"] = st["ks"], st["vs"]
    return o


def _plain_fork(st):
    R, B, K, L = (st["case"][k] for k in ("requests", "beams", "block", "layers"))
    o, C, S = st["outs"], st["rows"].shape[1], R * B
    old, lens, held = st["rows"].view(R, B, C), st["lens"].long().view(R, B), st["held"].long().view(R, B)
    parents = st["parents"].long()
    live, p = parents >= 0, parents.clamp(min=0)
    earlier = torch.ones((B, B), dtype=torch.bool, device=old.device).tril(-1)     # [i, j]: j in front of i
    first = ~((parents[:, :, None] == parents[:, None, :]) & earlier).any(2)
    ln, hd = lens.gather(1, p), held.gather(1, p)
    need, full = (ln + K - 1) // K, ln // K
    hd = torch.where(live, torch.where(first, hd, need), 0)
    take = live & ~first & (ln % K > 0)
    rank = (torch.cumsum(take.flatten(), 0) - 1).view(R, B)
    fresh = st["ring"][(st["state"][0] + rank.clamp(min=0)) % st["ring"].shape[0]]
    at = torch.arange(C, device=old.device)
    rows = old.gather(1, p[..., None].expand(-1, -1, C))
    listed_ = at < hd[..., None]
    split = take[..., None] & (at == full[..., None])
    source = rows.gather(2, full.clamp(max=C - 1)[..., None])[..., 0]
    rows = torch.where(split, fresh[..., None], rows)
    # old entries that no row lists any more, each page once, by request, entry and row
    had = at < held[..., None]
    kept = torch.zeros_like(had)
    again = torch.zeros_like(had)
    for i in range(B):
        kept |= (old == rows[:, i:i + 1]) & listed_[:, i:i + 1]
        again[:, i + 1:] |= (old[:, i + 1:] == old[:, i:i + 1]) & had[:, i:i + 1]
    back = (had & ~kept & ~again).permute(0, 2, 1).flatten()
    place = torch.cumsum(back, 0) - 1
    size = st["ring"].shape[0]
    longer = torch.cat([st["ring"], st["ring"][:1]])
    longer[torch.where(back, (st["state"][1] + place) % size, size)] = old.permute(0, 2, 1).flatten()
    st["ring"].copy_(longer[:size])
    o["block_tables_out"].copy_(torch.where(listed_, rows, o["block_tables_out"].view(R, B, C)).view(S, C))
    o["lens_out"].copy_(torch.where(live, ln, 0).flatten())
    o["held_out"].copy_(hd.flatten())
    o["ring_state_out"].copy_(st["state"] + torch.stack([take.sum(), back.sum()]))
    o["pairs"].copy_(torch.where(take[..., None], torch.stack([source, fresh], -1).long(), -1).view(S, 2))
    o["totals"].copy_(torch.stack([torch.zeros_like(take.sum()), live.sum(), take.sum(), back.sum()]))
    # the tokens of the partly filled pages; a row without a copy writes a page that it listed with what the page holds
    src, dst = o["pairs"][:, 0], o["pairs"][:, 1]
    t = torch.arange(K, device=old.device)
    moved = (src >= 0)[:, None] & (t < (o["lens_out"].long() % K)[:, None])
    a = torch.where(src >= 0, src, st["rows"][:, 0].long())[:, None] * K + t
    b = torch.where(moved, dst[:, None] * K + t, a).flatten()
    a = a.flatten()
    for name in ("kc", "vc") + (("ks", "vs") if st["case"]["pool"] == "int4" else ()):
        for layer in range(L):
            pages = st[name][layer]
            if name in ("ks", "vs"):
                pages[b // K, :, b % K] = pages[a // K, :, a % K]
            else:
                pages.flatten(0, 1)[b] = pages.flatten(0, 1)[a]
    return _fork_outputs(st)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "write":
        T, J, D = case["tokens"], case["kv"], case["dim"]
        e = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * (2 * J * (D * e + D // 2 + 4) + 8), "flops": 2 * T * J * D * 5}
    if case["op"] == "attn":
        S, g, H, J, D, K = (case[k] for k in ("seqs", "group", "heads", "kv", "dim", "block"))
        mean = (case["len_lo"] + case["len_hi"]) / 2
        own_len = (1 + case["own_hi"]) / 2 if g > 1 else 0
        tokens = S // g * mean + S * own_len if g > 1 else S * mean
        return {"bytes": tokens * J * (D + 8) + S * H * D * 4 + S * (mean + own_len) / K * 4, "flops": 4 * S * (mean + own_len) * H * D}
    if case["op"] == "select":
        rows = case["requests"] * case["beams"]
        e = 4 if case["dtype"] == "float32" else 2
        return {"bytes": rows * (1 - case["over"]) * case["vocab"] * e + rows * 5 + case["requests"] * case["take"] * 13, "flops": rows * (1 - case["over"]) * case["vocab"] * 3}
    R, B, K, J, D = (case[k] for k in ("requests", "beams", "block", "kv", "dim"))
    entries = R * B * ((case["len_lo"] + case["len_hi"]) / 2 + case["own_hi"] / 2) / K
    row = J * (D // 2 + 4) if case["pool"] == "int4" else J * D * 2
    # about B / e beams are not kept, so that as many rows get a copy of half a page, read and written, K and V
    copies = R * (1 - case["over"]) * B * 0.33
    return {"bytes": entries * 8 + R * B * 40 + copies * case["layers"] * (K / 2) * row * 4, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits (whole numbers have none of their own)
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "fork":
        return None
    st = prepare(case, seed)
    return {"write": _exact_write, "attn": _exact_attn, "select": _exact_select}[case["op"]](case, st)


def _exact_write(case, st):
    # the scales, from the rounded offset; the offset is rounded down and the codes are whole numbers
    out = {}
    for n in ("k", "v"):
        x = st[n].double()
        low = x.min(2).values
        step = torch.exp2(torch.floor(torch.log2(low.abs().clamp(min=2.0 ** -126))) - 7)
        offset = torch.floor(low / step) * step
        s = torch.zeros(st[n + "s"].shape, dtype=torch.float64, device=DEV)
        page, at = st["slots"] // case["block"], st["slots"] % case["block"]
        s[page, :, at, 0] = (x.max(2).values - offset) / 15
        s[page, :, at, 1] = offset
        out[n], out[n + "_scales"] = None, s
    return out


def _exact_attn(case, st):
    S, H, J, D, K = (case[k] for k in ("seqs", "heads", "kv", "dim", "block"))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)

    def rows(codes, scales, slot):
        c = codes.flatten(0, 1)[slot].int()
        x = torch.empty((slot.shape[0], J, D), dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = (c % 16).double(), (c // 16).double()
        s = scales[slot // K, :, slot % K].double()
        return s[..., 1:2] + s[..., 0:1] * x

    for s, L in enumerate(st["lens"].tolist()):
        if L == 0:
            continue
        t = torch.arange(L, device=DEV)
        slot = st["rows"][s].long()[t // K] * K + t % K
        k, v = rows(st["kc"], st["ks"], slot), rows(st["vc"], st["vs"], slot)
        q = st["q"][s].double().view(J, H // J, D)
        w = torch.softmax(torch.einsum("jgd,tjd->jgt", q, k) * st["scale"], -1)
        out[s] = torch.einsum("jgt,tjd->jgd", w, v).reshape(H, D)
    return out


def _exact_select(case, st):
    R, B, V, N = (case[k] for k in ("requests", "beams", "vocab", "take"))
    best = torch.empty((R, N), dtype=torch.float64, device=DEV)
    for r in range(R):
        x = torch.log_softmax(st["logits"][r * B:(r + 1) * B].double(), 1) + st["scores"][r].double().unsqueeze(1)
        over = st["over"][r]
        each = torch.cat([x[~over].flatten(), st["scores"][r][over].double(), torch.full((N,), -math.inf, dtype=torch.float64, device=DEV)])
        best[r] = torch.topk(each, N).values
    return {"tokens": None, "parents": None, "scores": best, "finished": None}
