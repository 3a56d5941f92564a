"""The largest sizes of the step calls."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 4])
def test_as_many_token_rows_as_32_bits_count(ops, T):
    """The rows behind the step's 70 tokens are padding up to the last one, and
    what lies behind the last one is left alone."""
    positions = torch.full((T + 9,), 5, dtype=torch.int32, device=DEV)
    slots = torch.full((T + 9,), 5, dtype=torch.int64, device=DEV)
    tables = torch.full((2, 20), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(50, device=DEV).int()
    o = ops.step_tables(i32([0, 0]), i32([30, 40]), tables, i32([0, 0]), ring,
                        torch.tensor([0, 50], device=DEV), 4, 50, positions=positions[:T], slots=slots[:T])
    assert o["totals"].tolist() == [0, 70, 18, 0] and ops.get_device_error() == 0
    assert positions[:70].tolist() == list(range(30)) + list(range(40))
    assert slots[:70].tolist() == list(range(30)) + list(range(32, 72))
    for x in (positions, slots):
        assert int(x[70:T].max()) == -1 == int(x[70:T].min())
        assert (x[T:] == 5).all()
