"""Beam selection and forks: counts past 32 bits, batches without a request."""

import pytest
import torch

from tests.test_gpu_beam import ops    # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kw", [dict(num_select=2 ** 32 + 4), dict(num_select=2 ** 31), dict(num_select=4, eos_token=2 ** 32 + 2),
                                dict(num_select=4, eos_token=2 ** 31), dict(num_select=4, eos_token=-2 ** 32)])
def test_counts_past_32_bits_are_refused(ops, kw):
    logits, scores = torch.zeros((2, 50), device=DEV), torch.zeros((1, 2), device=DEV)
    with pytest.raises(ValueError):
        ops.beam_select(logits, scores, **kw)
