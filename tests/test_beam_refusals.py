"""Host-side refusals of the 4-bit writes, the beam selection and the forks:
checked before anything is launched; the pointers are never followed."""

import ctypes

import pytest
import torch

OK, BAD, UNSUPPORTED, SMALL = 0, 1, 2, 3
A = 4096


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    return o


def int4(ops, k=A, v=A):
    q = ops.KvQuant()
    q.format, q.k_token_scales, q.v_token_scales = 4, k, v
    return q


def write(ops, quant, **kw):
    a = dict(k=A, ks=256, v=A, vs=256, slots=A, T=3, kc=A, vc=A, nb=4, K=16, H=2, D=128, dt=1)
    a.update(kw)
    return ops._write_quant(*a.values(), None if quant is None else ctypes.byref(quant), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, k=None), OK), (dict(T=-1), BAD), (dict(D=96), UNSUPPORTED),
    (dict(D=256, ks=512, vs=512), UNSUPPORTED),
    (dict(k=None), BAD), (dict(slots=None), BAD), (dict(slots=A + 4), BAD), (dict(ks=255), BAD),
    (dict(vs=0), BAD), (dict(kc=A + 2), BAD), (dict(k=A + 1), BAD), (dict(dt=2), BAD), (dict(nb=0), BAD),
    (dict(K=0), BAD), (dict(H=0), BAD), (dict(nb=2**62), BAD), (dict(nb=2**52), BAD),
    (dict(T=2**30, H=1), UNSUPPORTED)])
def test_write(ops, kw, want):
    assert write(ops, int4(ops), **kw) == want


def test_write_description(ops):
    assert write(ops, None) == BAD
    assert write(ops, int4(ops, k=None)) == BAD and write(ops, int4(ops, v=A + 2)) == BAD
    q = int4(ops)
    q.format = 5
    assert write(ops, q) == BAD


def test_kv_quant_arguments(ops):
    with pytest.raises(ValueError):
        ops.kv_quant("int4")
    with pytest.raises(ValueError):
        ops.kv_quant("int4", k_token_scales=torch.zeros(1, 1, 16, 2, dtype=torch.bfloat16),
                     v_token_scales=torch.zeros(1, 1, 16, 2, dtype=torch.bfloat16))     # not on a GPU


def beam(ops, **kw):
    a = dict(logits=A, stride=100, scores=A, finished=None, R=2, B=3, V=100, N=4, eos=-1, tokens=A, parents=A,
             out=A, over=A, ws=A, ws_bytes=1 << 40, dt=1)
    a.update(kw)
    return ops._beam(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=0, logits=None), OK), (dict(R=-1), BAD), (dict(B=0), BAD), (dict(B=33), UNSUPPORTED),
    (dict(N=33), UNSUPPORTED), (dict(N=0), BAD), (dict(V=0), BAD), (dict(V=2**22 + 1), UNSUPPORTED),
    (dict(eos=100), BAD), (dict(eos=-2), BAD), (dict(finished=A), BAD), (dict(stride=99), BAD),
    (dict(logits=None), BAD), (dict(scores=None), BAD), (dict(tokens=None), BAD), (dict(parents=None), BAD),
    (dict(out=None), BAD), (dict(ws=None), BAD), (dict(ws=A + 16), BAD), (dict(logits=A + 1), BAD),
    (dict(tokens=A + 2), BAD), (dict(dt=2), BAD), (dict(R=2**26, B=32, V=2**22, stride=2**22), UNSUPPORTED)])
def test_beam(ops, kw, want):
    assert beam(ops, **kw) == want


def fork(ops, **kw):
    a = dict(parents=A, lens=A, held=A, shared=None, tables=A, width=8, ring=A, ring_size=64, state=A, R=2, B=4,
             K=16, tables_out=A, lens_out=A, held_out=A, state_out=A, pairs=A, totals=A, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    return ops._fork(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=0, parents=None), OK), (dict(R=-1), BAD), (dict(B=0), BAD), (dict(B=33), UNSUPPORTED),
    (dict(width=0), BAD), (dict(K=0), BAD), (dict(ring_size=0), BAD), (dict(R=2**20, B=32, width=64), UNSUPPORTED),
    (dict(R=2**31 - 1, B=32, width=2**30), UNSUPPORTED),
    (dict(width=2**24, R=1, B=1, K=16), UNSUPPORTED), (dict(width=2**20, K=2**12, R=1, B=1), UNSUPPORTED),
    (dict(parents=None), BAD), (dict(ring=None), BAD), (dict(pairs=None), BAD), (dict(totals=None), BAD),
    (dict(state=A + 4), BAD), (dict(pairs=A + 4), BAD), (dict(lens=A + 2), BAD), (dict(ws=None), BAD),
    (dict(ws=A + 128), BAD), (dict(ws_bytes=64), SMALL)])
def test_fork(ops, kw, want):
    assert fork(ops, **kw) == want


def copy(ops, quant=None, **kw):
    a = dict(kc=A, vc=A, pairs=A, lens=A, S=3, L=1, nb=4, K=16, H=2, D=128, dt=1)
    a.update(kw)
    return ops._fork_copy(*a.values(), None if quant is None else ctypes.byref(quant), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=0, kc=None), OK), (dict(S=-1), BAD), (dict(L=0), BAD), (dict(L=40000), UNSUPPORTED), (dict(nb=0), BAD),
    (dict(nb=2**55, L=1000), BAD), (dict(kc=None), BAD), (dict(pairs=None), BAD), (dict(pairs=A + 4), BAD),
    (dict(lens=A + 2), BAD), (dict(dt=3), BAD), (dict(quant=True, D=96), UNSUPPORTED),
    (dict(quant=True, vc=A + 1), BAD)])
def test_copy(ops, kw, want):
    kw = dict(kw)
    quant = int4(ops) if kw.pop("quant", False) else None
    assert copy(ops, quant, **kw) == want
