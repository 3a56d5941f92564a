"""Beam selection: the sums of rows with values far from zero."""

import pytest
import torch

from tests.test_gpu_beam import check_select, ops    # noqa: F401 (ops: fixture)

pytestmark = pytest.mark.gpu


# the logarithm of a row around these values is kept in two ways (65536 lies between)
@pytest.mark.parametrize("at", [-65536.0, 65536.0])
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** -7), (0.0, 1.0), (1.0, 1.0), (0.5, 0.25), (3.0, 0.0), (200.0, 4.0)])
@pytest.mark.parametrize("V", [9, 600, 3000, 70000])
def test_rows_on_both_sides(ops, V, low, high, at):
    # halves of a row, alternate values, one value below or above many
    rows = torch.full((4, V), at - low)
    rows[0, V // 2:] = at + high
    rows[1, ::2] = at + high
    rows[2, V - 1] = at + high
    rows[3] = at + high
    rows[3, V // 3] = at - low
    check_select(ops, rows, torch.zeros((4, 1)), 5)
    check_select(ops, rows, torch.tensor([[0.0, -1.0], [-2.0, 0.5]]), 7)
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("at", [-65536.0, 65536.0, -131072.0, 65000.0])
def test_random_rows_on_both_sides(ops, at):
    g = torch.Generator().manual_seed(5)
    rows = at + 3 * torch.randn((6, 40000), generator=g)
    check_select(ops, rows, -torch.rand((2, 3), generator=g), 8)
    assert ops.get_device_error() == 0
