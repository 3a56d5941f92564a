"""Softmax weights behind a shared prefix carry 14 bits or more.

The prefix part enters its weights as two bf16 terms, a weight off by less
than 2^-14 of itself; with the sums' float32 roundings (64 accumulations of a
product of 16 keys, each within 2^-22 of the sum's magnitude: 2^-16; the row
sum 2^-18; exponent and its argument 2^-19) the output is off by less than
2^-13 of A = sum_x w_x |v_x| / sum_x w_x besides its own rounding, 2^-8 of the
value, as long as the scores themselves are exact.
"""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_prefix import call, ops, problem, want  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [40, 300])
@pytest.mark.parametrize("D,K", [(128, 16), (64, 8)])
def test_values_that_cancel(ops, S, D, K):  # noqa: F811
    """Every other key has weight w = 0.78 .. 0.82 (another one for each
    sequence) and values -1.25, the others weight 1 and values 1: the sums
    almost cancel, and a weight's rounding is what is left."""
    prefix = 512
    pb = problem([prefix + 1] * S, [1] * S, 2, 1, D, K, prefix, seed=D)
    table = torch.from_numpy(pb["table"]).long()
    pb["kc"][:] = 0
    pb["vc"][:] = 1
    odd = torch.arange(K) % 2 == 1
    kp, vp = pb["kc"][table], pb["vc"][table]
    kp[:, odd, :, 0] = -1
    vp[:, odd] = -1.25
    pb["kc"][table], pb["vc"][table] = kp, vp
    w = torch.linspace(0.78, 0.82, 2 * S).view(S, 2)
    pb["q"].zero_()
    pb["q"][:, :, 0] = (-w.log() * D ** 0.5).to(torch.bfloat16)      # one product a score: exact
    got = as_f64(call(ops, pb))
    assert ops.get_device_error() == 0
    ref, a = want(pb)
    assert np.abs(ref).max() < 0.05 and a.min() > 1
    assert np.all(np.abs(got - ref) <= 2.0**-13 * a + 2.0**-8 * np.abs(ref))


def test_the_tolerance_of_the_other_attention_calls(ops):  # noqa: F811
    """2e-3 + 1e-2 |ref|, as for decode and prefill, on short prefixes."""
    for prefix in (16, 32, 48, 128):
        pb = problem([prefix + 1 + s % 3 for s in range(500)], [1] * 500, 8, 2, 128, 16, prefix, seed=prefix)
        got = as_f64(call(ops, pb))
        ref, _ = want(pb)
        assert np.all(np.abs(got - ref) <= 2e-3 + 1e-2 * np.abs(ref))
