"""Attention with queries (and outputs) off the boundaries that the tensor-core
kernels load from: the kernel that such a call is sent to, bit for bit."""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64, check_attention
from tests.test_gpu_int4 import make, on_gpu
from oracle import quant as Q
from tests._helpers import storage

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def shifted(t, elements):
    """The same values, contiguous, ``elements`` behind a 256-byte boundary."""
    buf = torch.zeros(t.numel() + elements, dtype=t.dtype, device=DEV)
    view = buf[elements:].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 256 == elements * t.element_size() % 256
    return view


# elements off a 16-byte boundary; from which ones each format's tensor-core kernel loads
STEP = dict(bf16=2, k16v8=2, fp8=4, int8=4, int4=8)


@pytest.mark.parametrize("off", [1, 2, 3, 4, 5, 6, 8, 12])
def test_int4(ops, off):
    c = make([40, 300, 0, 1], 16, 4, 128, 16, torch.bfloat16, seed=off)
    q, kc, vc, ks, vs, bt, lens = c
    g = on_gpu(ops, c)
    kernel = 1 if off % STEP["int4"] == 0 else 2
    want = ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=300, kernel=kernel)
    out = torch.empty(q.numel() + off, dtype=q.dtype, device=DEV)[off:].view(q.shape)
    for share in (False, True):
        ops.paged_attention_decode_quant(shifted(g[0], off), *g[1:5], 0.1, g[5], max_context_len=300,
                                         out=out, share_prefix=share)
        assert ops.get_device_error() == 0
        ref = Q.paged_attention_decode_int4(storage(q), kc, vc, ks, vs, bt, lens, 0.1, "bf16")
        check_attention(as_f64(out), ref, "bf16")
        if not share:
            assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["bf16", "k16v8", "fp8", "int8"])
@pytest.mark.parametrize("off", [1, 2, 3, 4, 6, 8])
def test_other_formats(ops, fmt, off):
    gen = torch.Generator(device=DEV).manual_seed(off)
    nb, K, H, D, S = 30, 16, 2, 128, 3
    x = torch.randn((2, nb, K, H, D), generator=gen, device=DEV)
    q = torch.randn((S, 4 * H, D), generator=gen, device=DEV).to(torch.bfloat16)
    bt = torch.randperm(nb, generator=gen, device=DEV)[:S * 8].view(S, 8).to(torch.int32)
    lens = torch.tensor([128, 1, 77], dtype=torch.int32, device=DEV)
    codes = (x * 20).round().clamp(-127, 127).to(torch.int8)
    if fmt == "bf16":
        def run(q, out=None, kernel=0):
            return ops.paged_attention_decode(q, x[0].to(torch.bfloat16), x[1].to(torch.bfloat16), bt, lens, 0.1,
                                              max_context_len=128, out=out, kernel=kernel)
    else:
        s = torch.full((nb * K,), 0.05, device=DEV)
        qd = ops.kv_quant("int8", k_token_scales=s, v_token_scales=s.clone()) if fmt == "int8" else \
            ops.kv_quant(fmt, 0.05, 0.05)
        kc = x[0].to(torch.bfloat16) if fmt == "k16v8" else codes[0] if fmt == "int8" else \
            (x[0] * 20).to(torch.float8_e4m3fn)
        vc = codes[1] if fmt == "int8" else (x[1] * 20).to(torch.float8_e4m3fn)

        def run(q, out=None, kernel=0):
            return ops.paged_attention_decode_quant(q, kc, vc, bt, lens, 0.1, qd, max_context_len=128, out=out,
                                                    kernel=kernel)
    want = run(q, kernel=1 if off % STEP[fmt] == 0 else 2)
    out = torch.empty(q.numel() + 1, dtype=q.dtype, device=DEV)[1:].view(q.shape)
    assert torch.equal(run(shifted(q, off), out), want)
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("D,new", [(128, [200, 1, 77]), (64, [65, 130, 9]), (128, [17, 20, 30])])
def test_prefill(ops, D, new):
    gen = torch.Generator(device=DEV).manual_seed(D + new[0])
    nb, K, H, S = 64, 16, 2, len(new)
    kc, vc = (torch.randn((nb, K, H, D), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    T = sum(new)
    q = torch.randn((T, 4 * H, D), generator=gen, device=DEV).to(torch.bfloat16)
    cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=DEV)
    lens = torch.tensor([n + 50 for n in new], dtype=torch.int32, device=DEV)
    bt = torch.randperm(nb, generator=gen, device=DEV)[:S * 16].view(S, 16).to(torch.int32)

    def run(q, out=None, **kw):
        return ops.paged_attention_prefill(q, kc, vc, bt, cu, lens, 0.1, max(new), 256, out=out, **kw)
    want = run(q, kernel=2, num_splits=1)
    for qo, oo in ((2, 0), (0, 2), (6, 4), (8, 8)):
        out = torch.zeros(q.numel() + oo, dtype=q.dtype, device=DEV)[oo:].view(q.shape)
        run(shifted(q, qo), out)
        if (qo, oo) == (8, 8):
            assert torch.equal(out, run(q))
        else:
            assert torch.equal(out, want)
    assert ops.get_device_error() == 0
