"""Attention over 4-bit pages: scores keep a float32 sum's digits where a few
channels of the queries are far larger than the others."""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_int4 import ops    # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16_words(scale, offset):
    return torch.stack([torch.full((), scale), torch.full((), offset)]).to(torch.bfloat16)


@pytest.mark.parametrize("large", [(2, 40, 76, 102), (1, 41, 79, 127), (0, 3, 64, 125)])
@pytest.mark.parametrize("H_q,H_kv,share", [(8, 2, False), (8, 1, False), (4, 2, False), (8, 2, True), (7, 1, True)])
def test_two_keys_alike(ops, H_q, H_kv, share, large):
    # Two keys that differ in all channels but the four where the queries are large, values
    # -1 and 1: the output is tanh of half the scores' difference, whatever their size.
    rng = np.random.default_rng(H_q * 10 + H_kv)
    S, D, K, scale = 64, 128, 16, 8.0
    q = 0.004 * rng.standard_normal((S, H_q, D))
    codes = rng.integers(0, 16, (S, 2, H_kv, D))                           # [S, 2 tokens, H_kv, D]
    for c in large:
        q[..., c] = 100 * rng.choice([-1, 1], (S, H_q))
        codes[:, 1, :, c] = codes[:, 0, :, c]
    q = torch.from_numpy(q).to(torch.bfloat16)
    kc = torch.zeros((S, K, H_kv, D // 2), dtype=torch.uint8)
    kc[:, :2] = torch.from_numpy((codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8))
    ks = bf16_words(1.0, -7.5).expand(S, H_kv, K, 2).contiguous()
    vc = torch.zeros_like(kc)
    vs = bf16_words(1.0, -1.0).repeat(S, H_kv, K, 1)
    vs[:, :, 1, 1] = 1.0
    bt = torch.arange(S, dtype=torch.int32)[:, None]
    lens = torch.full((S,), 2, dtype=torch.int32)
    g = [t.to(DEV) for t in (q, kc, vc, bt, lens)]
    qd = ops.kv_quant("int4", k_token_scales=ks.to(DEV), v_token_scales=vs.to(DEV))
    out = as_f64(ops.paged_attention_decode_quant(*g, scale, qd, max_context_len=2, kernel=1, share_prefix=share))
    assert ops.get_device_error() == 0
    q64 = as_f64(q)
    G = H_q // H_kv
    delta = np.repeat((codes[:, 1] - codes[:, 0]).astype(np.float64), G, 1)
    delta = scale * (q64 * delta).sum(-1)
    assert np.abs(out - np.tanh(delta / 2)[..., None]).max() < 2            # (finite)
    # A score's error: eight steps of the product add 17 terms each, cut at 2^-23 of the
    # largest exponent among them (as measured by Fasi, Higham, Mikaitis and Pranesh,
    # "Numerical behavior of NVIDIA tensor cores", 2021).  Codes of the second pairs stand
    # below the normal f16 numbers and count as 64 there, so that exponent is 64 |q|'s, or
    # that of a partial sum, which is not above 400 x 15: 2^12 both times.  Cuts spread evenly
    # over a step 2^-11: 2^-11 sqrt(8 x 17 / 12) a score, the root of two more for two scores;
    # half as much again for cuts that are not independent.  An output is off by bf16's half
    # step, at most 2^-8 of its size below 0.64 (|delta| < 1.5), tanh's slope is above 0.29.
    near = np.abs(delta) < 1.5
    got = 2 * np.arctanh(np.clip(out, -0.99, 0.99)).mean(-1)
    rms = np.sqrt(((got - delta)[near] ** 2).mean())
    assert near.sum() > 50
    assert rms <= scale * 1.5 * 2 ** 0.5 * 2.0 ** -11 * (8 * 17 / 12) ** 0.5 + 0.64 * 2.0 ** -8 / 0.29, rms
