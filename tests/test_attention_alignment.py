"""Queries off the boundaries that the tensor-core kernels load from: refused on
the host where such a kernel is asked for, sent to the others where it is not.
The pointers are never followed."""

import ctypes

import pytest

BAD, UNSUPPORTED, SMALL = 1, 2, 3
A = 4096


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    return o


def quant(ops, fmt):
    if fmt == "bf16":
        return None
    q = ops.KvQuant()
    q.format = dict(fp8=1, int8=2, k16v8=3, int4=4)[fmt]
    q.k_scale = q.v_scale = 1.0
    q.k_token_scales = q.v_token_scales = A
    return ctypes.byref(q)


def decode(ops, fmt, q=A, out=A, kernel=0, ws=A, tables=A, lens=A, D=128):
    cfg = ops.AttentionConfig()
    cfg.kernel = kernel
    qd = quant(ops, fmt)
    # a long context, no workspace: the CUDA-core plan ends at the workspace check
    a = [q, A, A, tables, 64, lens, 1024, 3, 8, 2, D, 16, 4, 0.1, out, ws, 0 if ws == A else 1 << 40, 1]
    if qd is None:
        return ops._attention(*a, ctypes.byref(cfg), None)
    return ops._attention_quant(*a, qd, ctypes.byref(cfg), None)


@pytest.mark.parametrize("fmt,off", [("bf16", 2), ("k16v8", 2), ("fp8", 2), ("fp8", 4), ("int8", 4), ("int8", 12),
                                     ("int4", 2), ("int4", 4), ("int4", 8), ("int4", 24)])
def test_decode(ops, fmt, off):
    assert decode(ops, fmt, q=A + off, kernel=1) == UNSUPPORTED
    assert decode(ops, fmt, q=A + off) == SMALL                   # the CUDA-core plan
    assert decode(ops, fmt, q=A + 1, kernel=2, ws=2 * A) == BAD   # not even an element


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4"])
def test_tables_and_lengths(ops, fmt):
    for kw in (dict(tables=A + 2), dict(lens=A + 1)):
        assert decode(ops, fmt, kernel=2, ws=2 * A, **kw) == BAD


def prefill(ops, q=A, out=A, kernel=0, n=200, tables=A, cu=A):
    cfg = ops.AttentionConfig()
    cfg.kernel = kernel
    return ops._prefill(q, A, A, tables, 64, cu, A, 3, 3 * n, n, 1024, 8, 2, 128, 16, 4, 0.1, out, A, 0, 1,
                        ctypes.byref(cfg), None)


def test_prefill(ops):
    for kw in (dict(q=A + 4), dict(out=A + 8), dict(q=A + 8, out=A + 4)):
        assert prefill(ops, kernel=1, **kw) == UNSUPPORTED
    for kw in (dict(q=A + 2), dict(out=A + 2), dict(tables=A + 2), dict(cu=A + 2)):
        assert prefill(ops, **kw) == BAD
