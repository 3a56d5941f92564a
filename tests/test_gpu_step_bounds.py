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


def test_counts_past_32_bits_are_refused(ops):
    """An int32 argument must not take the low half of a larger count."""
    big = 2**32 + 4
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros((8, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    rows = torch.arange(8, device=DEV).int().view(1, 8)
    args = (q, pool, pool, rows[0], rows, i32([40]), 0.1)
    ops.paged_attention_decode_prefix(*args, prefix_len=32, max_context_len=128)
    for kw in (dict(prefix_len=32, max_context_len=big), dict(prefix_len=32, max_context_len=128, max_query_len=big),
               dict(prefix_len=-big, max_context_len=128)):
        with pytest.raises(ValueError):
            ops.paged_attention_decode_prefix(*args, **kw)
    with pytest.raises(ValueError):
        ops.prefix_workspace_bytes(1, 1, 1, big, 32, 2, 1, 64, 16, torch.bfloat16)
    with pytest.raises(ValueError):
        ops.step_tables(i32([0]), i32([3]), rows.clone(), i32([0]), i32([1, 2]), torch.tensor([0, 2], device=DEV),
                        big, 8, num_tokens=4)
    f = torch.ones((1, 8), device=DEV)
    with pytest.raises(ValueError):
        ops.verify_draft_tokens(f, None, i32([0]), f[0, :1], i32([0, 1]), big, out_tokens=i32([[0]]), num_new=i32([0]))
    assert ops.get_device_error() == 0
