"""Values behind the rotation go through as they are: an infinity or a NaN
there reaches no other value, and a zero keeps its sign.  Rows on 16-byte
boundaries and rows off them take different kernels."""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_rope import near, ops, problem, run, views, want_rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot", [(128, 0), (128, 64), (64, 32), (64, 0), (128, 16), (256, 128)])
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_behind_the_rotation(ops, D, rot, gap, interleaved, dtype):  # noqa: F811
    pb = problem(6, 4, 2, D, 4, rot, dtype, seed=D + rot, gap=gap)
    rows = pb["qkv"][:, :(4 + 2) * D].view(6, 6, D)         # query and key heads
    rng = np.random.default_rng(rot)
    special = [float("inf"), float("-inf"), float("nan"), -0.0, 0.0]
    for t in range(6):
        for h in range(6):
            for x in rng.choice(np.arange(rot, D), 6, replace=False):
                rows[t, h, x] = special[int(rng.integers(5))]
    out, kc, _, _ = run(ops, pb, dtype, False, interleaved)
    assert ops.get_device_error() == 0
    q, k, _ = views(pb, pb["qkv"])
    k_got = kc.view(-1, 2, D)[torch.from_numpy(pb["slots"]).to(kc.device)]
    for what, x, got in (("q", as_f64(q), as_f64(out)), ("k", as_f64(k), as_f64(k_got))):
        a, b = x[..., rot:], got[..., rot:]
        assert np.array_equal(a, b, equal_nan=True), what
        zero = a == 0
        assert np.array_equal(np.signbit(a[zero]), np.signbit(b[zero])), what
        x = x.copy()
        x[..., rot:] = 0
        ref, mag = want_rows(pb, x, None, interleaved)
        near(got[..., :rot], ref[..., :rot], mag[..., :rot], dtype, what)
