"""Norm and rotation in front of a write into 4-bit pages: through plain pools that
hold the step's tokens one after the other."""

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests._helpers import storage
from tests.test_gpu_int4 import empty_pool, ops, same_pool    # noqa: F401 (ops: fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,J,H,D,K", [(1, 2, 8, 128, 16), (37, 8, 32, 128, 16), (130, 3, 6, 64, 8)])
def test_rotated_rows(ops, T, J, H, D, K, dtype):
    rng = np.random.default_rng(T)
    gen = torch.Generator(device=DEV).manual_seed(T)
    qkv = torch.randn((T, (H + 2 * J) * D), generator=gen, device=DEV).to(dtype)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, J * D, J * D], 1))
    weight = torch.rand(D, generator=gen, device=DEV).to(dtype)
    turn = torch.randn((300, D), generator=gen, device=DEV)
    positions = torch.randint(0, 300, (T,), generator=gen, device=DEV, dtype=torch.int32)
    nb = -(-T // K) + 3
    slots = torch.from_numpy(rng.permutation(nb * K)[:T].astype(np.int64)).to(DEV)
    # a plain cache, for the values
    plain = [torch.zeros((nb, K, J, D), dtype=dtype, device=DEV) for _ in range(2)]
    want_q = ops.paged_qk_norm_rope_append(q, k, v, positions, slots, *plain, turn, weight, weight)
    step = [torch.zeros((-(-T // K), K, J, D), dtype=dtype, device=DEV) for _ in range(2)]
    got_q = ops.paged_qk_norm_rope_append(q, k, v, positions, torch.arange(T, device=DEV), *step, turn, weight, weight)
    rows = [x.flatten(0, 1)[:T] for x in step]
    kc, ks = empty_pool(nb, K, J, D, rng)
    vc, vs = empty_pool(nb, K, J, D, rng)
    d = [t.to(DEV) for t in (kc, vc, ks, vs)]
    quant = ops.kv_quant("int4", k_token_scales=d[2], v_token_scales=d[3])
    ops.paged_kv_write_quant(*rows, slots, d[0], d[1], quant)
    assert ops.get_device_error() == 0
    assert torch.equal(got_q, want_q)
    for x, y in zip(rows, plain):
        assert torch.equal(x, y.flatten(0, 1)[slots])
    want = Q.kv_write_int4(kc.numpy(), vc.numpy(), storage(ks), storage(vs), *(r.float().cpu().numpy() for r in rows),
                           slots.cpu().numpy())
    same_pool(d[0], d[2], want[0], want[2])
    same_pool(d[1], d[3], want[1], want[3])
    with pytest.raises(ValueError, match="plain pools"):
        ops.paged_qk_norm_rope_append(q, k, v, positions, slots, d[0], d[1], turn, quant=quant)
