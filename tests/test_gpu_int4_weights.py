"""Attention over 4-bit pages: sums keep their digits where thousands of rows add up to
little."""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_int4 import ops    # noqa: F401 (fixture)
from tests.test_gpu_int4_scores import bf16_words

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_sum_of_many_rows(ops):
    # Means of 131072 rows by one CTA a head group, small beside their terms: what the sums
    # lose must not lean to one side.  An output may be off by its own rounding, the mean
    # of 1024 of them by 2^-8 / sqrt(12) / 32 of their size; five times that.
    rng = np.random.default_rng(1)
    T, H, D, K = 131072, 8, 128, 64
    kb, vb = (rng.integers(0, 256, (T // K, K, H, D // 2), dtype=np.uint8) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((1, H, D))).to(torch.bfloat16)
    want = np.empty((H, D))
    for h in range(H):
        k, v = (np.stack([b[:, :, h] & 15, b[:, :, h] >> 4], -1).reshape(T, D) - 7.5 for b in (kb, vb))
        p = np.exp(0.01 * (k @ as_f64(q)[0, h]))
        want[h] = p @ v / p.sum()
    words = bf16_words(0.25, -1.875).to(DEV).repeat(T // K, H, K, 1)
    qd = ops.kv_quant("int4", k_token_scales=words, v_token_scales=bf16_words(1.0, -7.5).to(DEV).repeat(T // K, H, K, 1))
    bt = torch.arange(T // K, dtype=torch.int32, device=DEV)[None]
    out = as_f64(ops.paged_attention_decode_quant(q.to(DEV), torch.from_numpy(kb).to(DEV), torch.from_numpy(vb).to(DEV), bt,
                                                  torch.tensor([T], dtype=torch.int32, device=DEV), 0.04, qd,
                                                  max_context_len=T, kernel=1, num_splits=1))[0]
    assert ops.get_device_error() == 0
    size = np.sqrt((want ** 2).mean())
    assert size < 0.1
    assert abs((out - want).mean()) <= 5 * size * 2.0 ** -8 / 12 ** 0.5 / 32
