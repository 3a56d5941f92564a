"""Attention over 4-bit pages: what one query head or one beam holds changes no
other head's and no other beam's result."""

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests._helpers import as_f64, check_attention, storage
from tests.test_gpu_int4 import make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def others_hold(ops, c, row, head, kernel, share):
    """The rows but (row, head) against the oracle without that row's values."""
    q, kc, vc, ks, vs, bt, lens = c
    g = on_gpu(ops, c)
    out = ops.paged_attention_decode_quant(*g[:5], 128 ** -0.5, g[5], max_context_len=int(lens.max()),
                                           kernel=kernel, share_prefix=share)
    assert ops.get_device_error() == 0
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[row, head] = False
    clean = torch.where(keep[..., None], q, torch.zeros_like(q))
    ref = Q.paged_attention_decode_int4(storage(clean), kc, vc, ks, vs, bt, lens, 128 ** -0.5, "bf16")
    check_attention(as_f64(out)[keep.numpy()], ref[keep.numpy()], "bf16")
    return as_f64(out)[row, head]


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 1e30, -3e38, 1e-38])
@pytest.mark.parametrize("H_q,H_kv,group", [(8, 2, 1), (16, 2, 1), (8, 2, 4), (7, 1, 2), (8, 1, 2), (5, 1, 3), (3, 1, 2)])
def test_one_row(ops, H_q, H_kv, group, value, kernel):
    lens = [130, 90, 64, 77][:max(2, group)]
    for row, head, every in ((0, 1, False), (1, 0, True), (0, H_q - 1, False)):
        c = make(lens, H_q, H_kv, 128, 16, torch.bfloat16, seed=H_q + row, share=3, group=group)
        if every:
            c[0][row, head] *= value
        else:
            c[0][row, head, 5] = value
        got = others_hold(ops, c, row, head, kernel, group > 1)
        if not np.isfinite(value):
            assert np.isnan(got).all()      # as the softmax of scores that are not numbers


def test_heads_of_very_different_sizes(ops):
    # each head's own tolerance: sizes from 2^-60 to 2^60 with a scale for the largest
    lens = [300, 40]
    c = make(lens, 8, 1, 128, 16, torch.bfloat16, seed=3)
    for scale, sizes in ((2.0 ** -63, [60, 59, 0, -60, 30, 58, 60, 1]), (2.0 ** 57, [-60, -61, -100, -62, -59, -80, -60, -64])):
        q = c[0].clone() * torch.tensor([2.0 ** e for e in sizes])[:, None].to(torch.bfloat16)
        cc = (q, *c[1:])
        g = on_gpu(ops, cc)
        out = ops.paged_attention_decode_quant(*g[:5], scale, g[5], max_context_len=300, kernel=1)
        ref = Q.paged_attention_decode_int4(storage(q), *c[1:5], c[5], c[6], scale, "bf16")
        check_attention(as_f64(out), ref, "bf16")
