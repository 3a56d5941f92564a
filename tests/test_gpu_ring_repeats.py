"""Kernels that read a ring of stages: the same call again gives the same bits, with
warps that lag behind others (rows of very different lengths, padding)."""

import numpy as np
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


@pytest.mark.parametrize("D,K,new", [(128, 16, [1, 40, 7, 64]), (64, 8, [33, 2, 64]), (128, 32, [16] * 5)])
def test_prefill(ops, D, K, new):
    gen = torch.Generator(device=DEV).manual_seed(D + K)
    lens = [n + 37 * i for i, n in enumerate(new)]
    lens[0] += 1500
    wide = -(-max(lens) // K)
    S, H, nb = len(new), 2, wide * len(new)
    kc, vc = (torch.randn((nb, K, H, D), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((sum(new), 4 * H, D), generator=gen, device=DEV).to(torch.bfloat16)
    cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=DEV)
    cl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    bt = torch.randperm(nb, generator=gen, device=DEV).view(S, wide).to(torch.int32)
    first = ops.paged_attention_prefill(q, kc, vc, bt, cu, cl, 0.1, max(new), max(lens), kernel=2)
    for _ in range(60):
        assert torch.equal(ops.paged_attention_prefill(q, kc, vc, bt, cu, cl, 0.1, max(new), max(lens), kernel=2), first)
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotation(ops, dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    T, H, J, D, K = 4001, 12, 3, 128, 16
    qkv = torch.randn((T, (H + 2 * J) * D), generator=gen, device=DEV).to(dtype)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, J * D, J * D], 1))
    weight = torch.rand(D, generator=gen, device=DEV).to(dtype)
    turn = torch.randn((500, D), generator=gen, device=DEV)
    positions = torch.randint(-200, 500, (T,), generator=gen, device=DEV, dtype=torch.int32)
    nb = -(-T // K) + 1
    slots = torch.randperm(nb * K, generator=gen, device=DEV)[:T].contiguous()
    slots[::7] = -1

    def run():
        pools = [torch.zeros((nb, K, J, D), dtype=dtype, device=DEV) for _ in range(2)]
        out = torch.zeros((T, H, D), dtype=dtype, device=DEV)
        ops.paged_qk_norm_rope_append(q, k, v, positions, slots, *pools, turn, weight, weight, q_out=out)
        return out, *pools
    first = run()
    for _ in range(30):
        for x, y in zip(run(), first):
            assert torch.equal(x, y)
    assert ops.get_device_error() == 0
