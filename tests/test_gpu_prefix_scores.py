"""Scores at the ends of the float32 range behind a shared prefix.

Tolerance as in test_gpu_prefix_weights.py: the scores here are equal for all
keys that weigh anything.
"""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_prefix import call, ops, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def test_scores_of_minus_infinity_in_front(ops):  # noqa: F811
    """A first tile whose scores overflow to -inf weighs nothing, however low
    the scores behind it are."""
    prefix = 384
    pb = problem([prefix + 3] * 6, [1] * 6, 2, 1, 128, 16, prefix, seed=8)
    table = torch.from_numpy(pb["table"]).long()
    pb["q"].fill_(0)
    pb["q"][:, :, :2] = 1e10
    kp = pb["kc"][table].view(prefix, 1, 128)
    kp[:128, :, :2] = -3e38
    kp[128:, :, :2] = -1.5e-7                    # -3e3 * scale: weights far below 2^-149 of e^0
    pb["kc"][table] = kp.view(-1, 16, 1, 128)
    own = torch.ones(pb["kc"].shape[0], dtype=torch.bool)
    own[table] = False
    pb["kc"][own] = pb["kc"][own].nan_to_num(0)
    pb["kc"][own, :, :, :2] = -1.5e-7
    pb["vc"][own] = pb["vc"][own].nan_to_num(0)
    got = as_f64(call(ops, pb))
    assert ops.get_device_error() == 0
    # equal weights over all keys but the first 128
    vc = pb["vc"].double().view(-1, 128)
    for s in range(6):
        at = torch.tensor([int(pb["full"][s, x // 16]) * 16 + x % 16 for x in range(128, prefix + 3)])
        ref, a = vc[at].mean(0).numpy(), vc[at].abs().mean(0).numpy()
        assert np.all(np.abs(got[s] - ref) <= 2.0**-13 * a + 2.0**-8 * np.abs(ref)), s
