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


def test_forks_without_a_group(ops):
    ring = torch.arange(20, dtype=torch.int32, device=DEV)
    state = torch.tensor([3, 17], device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    kw = dict(ring_state_out=torch.full((2,), -9, device=DEV), totals=torch.full((4,), -9, dtype=torch.int32, device=DEV))
    for given in ({}, kw):
        got = ops.fork_tables(none.view(0, 4), none, none, none.view(0, 6), ring, state, 16, **given)
        assert got["ring_state_out"].tolist() == [3, 17] and got["totals"].tolist() == [0] * 4
        assert got["lens_out"].shape == (0,) and got["pairs"].shape == (0, 2)
    assert ring.tolist() == list(range(20)) and ops.get_device_error() == 0
