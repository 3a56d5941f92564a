"""Shared-prefix groups over 4-bit pages: where they are taken, and where the mode is
ignored."""

import pytest
import torch

from tests.test_gpu_int4 import check, make, on_gpu, ops    # noqa: F401 (ops: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H_q,H_kv", [(5, 1), (12, 2), (7, 1), (16, 2)])
def test_ignored_above_four_heads(ops, H_q, H_kv):
    c = make([300, 310, 290, 5, 0, 640], H_q, H_kv, 128, 16, torch.bfloat16, seed=H_q, share=17, group=2)
    a = check(ops, c, 128 ** -0.5, share_prefix=True)
    assert torch.equal(a, check(ops, c, 128 ** -0.5))
    sizes = (6, H_q, H_kv, 128, 16, 640, torch.bfloat16, on_gpu(ops, c)[5])
    assert ops.attention_quant_workspace_bytes(*sizes, share_prefix=True) == ops.attention_quant_workspace_bytes(*sizes)


@pytest.mark.parametrize("B", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("H_q,H_kv", [(2, 2), (4, 2), (3, 1), (8, 2)])
def test_any_number_of_beams(ops, H_q, H_kv, B):
    # groups that hold rows of one request, of several, and a last one that is not full
    lens = [100 + 16 * (i // B) + i % 3 for i in range(3 * B + 1)]
    c = make(lens, H_q, H_kv, 128, 16, torch.bfloat16, seed=B, share=6, group=B)
    check(ops, c, 128 ** -0.5, share_prefix=True)
