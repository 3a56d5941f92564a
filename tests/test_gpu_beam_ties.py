"""Beam selection: rows alike give candidates alike, wherever the rows lie."""

import pytest
import torch

from tests.test_gpu_beam import check_select, ops    # noqa: F401 (ops: fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 3, 15, 700, 701, 999, 2049, 5003, 16385, 50021])
def test_beams_alike(ops, V, dtype):
    # the same row for every beam, the same score for some: the lowest beam goes first
    g = torch.Generator().manual_seed(V)
    row = (3 * torch.randn((2, 1, V), generator=g)).to(dtype)
    logits = row.expand(2, 7, V).reshape(14, V)
    scores = torch.tensor([[-1.0] * 7, [-2.0, -1.0, -1.0, -3.0, -1.0, -2.0, -1.0]])
    check_select(ops, logits, scores, 21)
    logits = torch.full((14, V), -0.75, dtype=dtype)
    logits[:, V - 1] = 1.5
    logits[:, V // 3] = 1.5
    check_select(ops, logits, scores, 30)
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [5, 1000, 4096, 33001])
def test_any_address(ops, V, dtype):
    # bit for bit, at every distance from a 16-byte boundary; neighbours hold larger values
    g = torch.Generator().manual_seed(V)
    logits = (3 * torch.randn((4, V), generator=g)).to(dtype).to(DEV)
    scores = -torch.rand((2, 2), generator=g).to(DEV)
    want = ops.beam_select(logits, scores, 9)
    for lead in range(16 // logits.element_size()):
        for pad in (0, 5):
            wide = torch.full((4, lead + V + pad), 80.0, dtype=dtype, device=DEV)
            wide[:, lead:lead + V] = logits
            for x, y in zip(ops.beam_select(wide[:, lead:lead + V], scores, 9), want):
                assert torch.equal(x, y)
