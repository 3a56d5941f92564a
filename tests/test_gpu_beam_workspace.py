"""Beam selection: the workspace of a batch serves every smaller one."""

import pytest
import torch

from tests.test_gpu_beam import check_select, ops, rand    # noqa: F401 (ops: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,V,N", [(8, 131072, 8), (4, 32000, 8), (5, 50021, 10), (1, 1000, 32), (32, 700, 32), (3, 2 ** 22, 4)])
def test_bytes_never_fall(ops, B, V, N):
    most = 0
    for R in list(range(0, 200)) + [511, 512, 513]:
        need = ops.beam_select_workspace_bytes(R, B, V, N)
        assert need >= most
        most = need
    for R, b, n in ((40, max(1, B - 1), N), (40, B, max(1, N // 2)), (3, max(1, B // 2), N)):
        assert ops.beam_select_workspace_bytes(R, b, V, n) <= ops.beam_select_workspace_bytes(R, B, V, N)


def test_smaller_batches_in_one_buffer(ops):
    B, V, N = 4, 32000, 8
    ws = torch.empty(ops.beam_select_workspace_bytes(45, B, V, N), dtype=torch.uint8, device="cuda")
    for R in (45, 37, 36, 20, 5, 1):
        for dtype in (torch.bfloat16, torch.float32):
            logits, scores = rand(R, B, V, dtype, seed=R)
            check_select(ops, logits, scores, N, workspace=ws)
    assert ops.get_device_error() == 0
