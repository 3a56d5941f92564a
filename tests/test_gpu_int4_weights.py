"""Attention over 4-bit pages: sums keep their digits where terms cancel (weights of
two keys) and where thousands of rows add up to little."""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_int4 import ops    # noqa: F401 (fixture)
from tests.test_gpu_int4_scores import bf16_words

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H_q,H_kv,K,share", [(8, 2, 16, False), (3, 1, 8, False), (8, 1, 16, False), (5, 1, 8, False),
                                              (8, 2, 16, True), (8, 8, 8, True), (7, 1, 16, True)])
def test_weights_of_two_keys(ops, H_q, H_kv, K, share):
    # Values 7 and -8 under weights of about 8 : 7.  The queries have one channel, so scores
    # are exact but for a rounding or two.
    rng = np.random.default_rng(H_q + K)
    S, D, scale, ch = 48, 128, 1.0, 21
    q = np.zeros((S, H_q, D))
    q[..., ch] = (np.log(8 / 7) + 0.01 * rng.standard_normal((S, H_q))) / 5
    q = torch.from_numpy(q).to(torch.bfloat16)
    kc = torch.zeros((S, K, H_kv, D // 2), dtype=torch.uint8)
    kc[:, 0, :, ch // 2] = 9 << 4                                           # codes 9 and 4: five apart
    kc[:, 1, :, ch // 2] = 4 << 4
    ks = bf16_words(1.0, -4.0).repeat(S, H_kv, K, 1)
    vc = torch.zeros_like(kc)
    vc[:, 0] = 0xFF                                                         # codes 15 and 0
    vs = bf16_words(1.0, -8.0).repeat(S, H_kv, K, 1)
    bt = torch.arange(S, dtype=torch.int32)[:, None]
    g = [t.to(DEV) for t in (q, kc, vc, bt, torch.full((S,), 2, dtype=torch.int32))]
    qd = ops.kv_quant("int4", k_token_scales=ks.to(DEV), v_token_scales=vs.to(DEV))
    out = as_f64(ops.paged_attention_decode_quant(*g, scale, qd, max_context_len=2, kernel=1, share_prefix=share))
    assert ops.get_device_error() == 0
    p0 = 1 / (1 + np.exp(-5 * as_f64(q)[..., ch]))
    want = (7 * p0 - 8 * (1 - p0))[..., None]
    assert 0.005 < np.abs(want).mean() < 0.1
    # the output's half step; weights of 7 + 8: two f16 numbers (2^-21), the exponential
    # (2^-22), a score's roundings (three of 2^-24 of less than 1) and six of sums
    assert (np.abs(out - want) <= np.abs(want) * 2.0 ** -8 + 15 * (2.0 ** -21 + 2.0 ** -22 + 9 * 2.0 ** -24)).all()


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
