"""Host-side refusals of the step calls (tables, norm + rotation + append,
attention behind a shared prefix, draft verification): checked before anything
is launched, so no GPU is needed; the pointers are never followed."""

import ctypes

import pytest

OK, BAD, UNSUPPORTED, SMALL = 0, 1, 2, 3
A = 4096                                  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    return o


def step(ops, **kw):
    a = dict(lens=A, counts=A, tables=A, width=4, held=A, shared=None, ring=A, ring_size=8,
             state=A, S=2, T=0, K=4, nb=8, ctx=A, cu=A, cb=A, pos=A, slots=A, held_out=A,
             state_out=A, totals=A)
    a.update(kw)
    return ops._step_tables(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), BAD), (dict(T=-1), BAD), (dict(K=0), BAD), (dict(width=0), BAD),
    (dict(ring_size=0), BAD), (dict(nb=0), BAD), (dict(lens=None), BAD), (dict(ring=None), BAD),
    (dict(T=3, slots=None), BAD), (dict(totals=None), BAD), (dict(state=A + 4), BAD),
    (dict(held=A + 2), BAD), (dict(width=2**30, K=4), UNSUPPORTED),
    (dict(S=2**20, width=2**12), UNSUPPORTED), (dict(nb=2**62, K=4), BAD)])
def test_step_tables(ops, kw, want):
    assert step(ops, **kw) == want


def rope(ops, quant=None, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, wq=None, wk=None, eps=1e-6, pos=A, cs=A,
             far=100, rot=64, inter=0, slots=A, T=3, H=8, J=2, D=64, out=A, os=512, kc=A, vc=A,
             nb=4, K=16, dt=1)
    a.update(kw)
    return ops._rope_append(*a.values(), None if quant is None else ctypes.byref(quant), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, q=None, k=None), OK), (dict(T=-1), BAD), (dict(rot=63), BAD), (dict(rot=66), BAD),
    (dict(rot=-2), BAD), (dict(inter=2), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(far=0), BAD), (dict(D=65, rot=0), UNSUPPORTED), (dict(D=514, rot=0), UNSUPPORTED),
    (dict(q=None), BAD), (dict(cs=None), BAD), (dict(slots=A + 4), BAD), (dict(q=A + 1), BAD),
    (dict(qs=511), BAD), (dict(vs=100), BAD), (dict(os=8), BAD), (dict(dt=2), BAD),
    (dict(nb=2**62), BAD), (dict(H=0), BAD)])
def test_rope(ops, kw, want):
    assert rope(ops, **kw) == want


def test_rope_quant(ops):
    q = ops.KvQuant()
    q.format = 7
    assert rope(ops, q) == BAD
    q.format, q.k_scale, q.v_scale = 1, 0.0, 1.0
    assert rope(ops, q) == BAD
    q.format = 2
    assert rope(ops, q) == BAD                       # no token scales
    q.k_token_scales, q.v_token_scales = A, A
    assert rope(ops, q, J=256, ks=16384, vs=16384) == UNSUPPORTED


def prefix(ops, **kw):
    a = dict(q=A, kc=A, vc=A, table=A, P=64, bt=A, width=16, cu=None, lens=A, S=4, T=4, mq=1,
             ml=200, H=8, J=2, D=128, K=16, nb=64, scale=0.1, out=A, ws=A, wb=2**40, dt=1)
    a.update(kw)
    return ops._prefix(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=0, T=0), OK), (dict(S=-1, T=-1), BAD), (dict(P=60), BAD), (dict(P=-16), BAD),
    (dict(T=5), BAD), (dict(mq=2), BAD), (dict(H=7), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(D=96), UNSUPPORTED), (dict(K=12, P=0), UNSUPPORTED),
    (dict(dt=0), UNSUPPORTED), (dict(H=32, J=2), UNSUPPORTED), (dict(cu=A, mq=3), UNSUPPORTED),
    (dict(S=4096, T=4096), UNSUPPORTED), (dict(q=None), BAD), (dict(table=None), BAD),
    (dict(q=A + 8), BAD), (dict(kc=A + 8), BAD), (dict(ws=A + 16), BAD), (dict(width=0), BAD),
    (dict(width=2**28), UNSUPPORTED), (dict(nb=2**30), UNSUPPORTED)])
def test_prefix(ops, kw, want):
    assert prefix(ops, **kw) == want


def verify(ops, **kw):
    a = dict(t=A, ts=100, d=A, dss=300, dts=100, tok=A, u=A, cu=A, S=2, T=6, mq=3, V=100, out=A,
             new=A, dt=0)
    a.update(kw)
    return ops._verify(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=0, t=None), OK), (dict(S=-1), BAD), (dict(T=-1), BAD), (dict(mq=0), BAD),
    (dict(V=0), BAD), (dict(V=2**22 + 1, ts=2**23), UNSUPPORTED), (dict(ts=99), BAD),
    (dict(dss=-1), BAD), (dict(t=None), BAD), (dict(out=None), BAD), (dict(tok=A + 2), BAD),
    (dict(t=A + 2), BAD), (dict(dt=5), BAD), (dict(S=2**28), UNSUPPORTED)])
def test_verify(ops, kw, want):
    assert verify(ops, **kw) == want


def test_cpu_tensors_are_refused(ops):
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        ops.step_tables(i, i, i.view(2, 1), i, i, i.long(), 4, 4, num_tokens=2)
    with pytest.raises(ValueError):
        ops.verify_draft_tokens(f, None, i, f[:, 0].contiguous(), i, 1)
    p = torch.zeros((2, 4, 1, 64))
    x = torch.zeros((2, 1, 64))
    with pytest.raises(ValueError):
        ops.paged_qk_norm_rope_append(x, x, x, i, i.long(), p, p, torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        ops.paged_attention_decode_prefix(x, p, p, i, i.view(2, 1), i, 1.0, 0, 4)
