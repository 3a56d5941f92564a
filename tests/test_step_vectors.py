"""The step calls take vectors as vectors: a table of the same number of values
is refused (checked on the host; no GPU is needed)."""

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    return o


@pytest.mark.parametrize("shape", [(4, 1), (1, 4), (2, 2), (1, 1, 4)])
def test_a_table_is_no_vector(ops, shape):
    dev = torch.zeros(1).get_device()
    flat = torch.zeros(4, dtype=torch.int32)
    assert ops._vec(flat, "lens", torch.int32, 4, dev) == flat.data_ptr()
    with pytest.raises(ValueError):
        ops._vec(torch.zeros(shape, dtype=torch.int32), "lens", torch.int32, 4, dev)
