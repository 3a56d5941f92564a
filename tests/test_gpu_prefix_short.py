"""Attention behind a shared prefix where sequences end before the prefix does.

Keys and values that a sequence does not see must not reach it, whatever they
hold: slots of the prefix that nobody has filled yet hold NaN here, and so do
filled ones that other sequences see.  Tolerances as in test_gpu_prefix.py.
"""

import numpy as np
import pytest
import torch

from tests._helpers import as_f64
from tests.test_gpu_prefix import call, check, ops, problem, want  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = "cuda"


def slot(pb, x):
    """(block, offset) of prefix token x."""
    return int(pb["table"][x // pb["K"]]), x % pb["K"]


def stale(pb, first, value=float("nan")):
    """Prefix tokens from `first` on hold `value`."""
    for x in range(first, pb["prefix"]):
        b, o = slot(pb, x)
        pb["kc"][b, o] = value
        pb["vc"][b, o] = value
    return pb


@pytest.mark.parametrize("lens", [[0, 1, 7, 64, 65, 100], [127, 128, 129, 191], [5], [0, 0, 0], [190] * 40])
@pytest.mark.parametrize("D,K", [(128, 16), (64, 8), (128, 48)])
def test_nobody_reaches_the_end_of_the_prefix(ops, lens, D, K):  # noqa: F811
    """The prefix is still being filled: what lies behind the longest sequence
    is stale, and so are the table entries there."""
    pb = stale(problem(lens, [1] * len(lens), 8, 2, D, K, 192, seed=K), max(lens))
    pb["table"][-(-max(lens) // K):] = 10**6
    out = call(ops, pb)
    assert all((out[s] == 0).all() for s, n in enumerate(lens) if n == 0)
    check(ops, pb, out)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("part", ["kc", "vc"])
@pytest.mark.parametrize("D,K", [(128, 16), (64, 8)])
def test_a_value_that_only_longer_sequences_see(ops, value, part, D, K):  # noqa: F811
    lens = [300, 0, 150, 149, 192, 151, 40, 191, 1000]
    pb = problem(lens, [1] * len(lens), 8, 2, D, K, 192, seed=D)
    b, o = slot(pb, 150)
    pb[part][b, o, :, 3:9] = value
    got = as_f64(call(ops, pb))
    assert ops.get_device_error() == 0
    clean = dict(pb, **{part: pb[part].clone()})
    clean[part][b, o] = 0
    ref, a = want(clean)
    for s, n in enumerate(lens):
        if n > 150:
            # (an infinite key may weigh nothing, as it would in one sequence)
            if part == "vc" or np.isnan(value):
                assert not np.isfinite(got[s][:, 3:9]).any()
            if part == "vc":
                assert np.isfinite(got[s][:, :3]).all() and np.isfinite(got[s][:, 9:]).all()
        else:
            tol = (2.0**-7 + 2.0**-8) * a[s] + 2.0**-8 * np.abs(ref[s])
            assert np.all(np.abs(got[s] - ref[s]) <= tol), s


@pytest.mark.parametrize("H,J,D,K,most", [(8, 8, 128, 16, 8), (8, 2, 64, 8, 2), (16, 8, 128, 32, 4), (32, 16, 128, 16, 2)])
def test_packed_new_tokens_around_the_end_of_the_prefix(ops, H, J, D, K, most):  # noqa: F811
    """New tokens that lie inside the prefix, at its end, across it and behind."""
    prefix = 160
    rng = np.random.default_rng(H)
    lens, news = [], []
    for n in range(1, most + 1):
        for first in (0, 1, 63, prefix - most - 1, prefix - 2, prefix - 1, prefix, prefix + 5):
            lens.append(first + n)
            news.append(n)
    order = rng.permutation(len(lens))
    lens, news = [lens[i] for i in order], [news[i] for i in order]
    pb = problem(lens, news, H, J, D, K, prefix, seed=H)
    pb["single"] = False
    check(ops, pb)
    short = [(n, m) for n, m in zip(lens, news) if n < prefix]
    pb = stale(problem([n for n, _ in short], [m for _, m in short], H, J, D, K, prefix, seed=H + 1),
               max(n for n, _ in short))
    pb["single"] = False
    check(ops, pb)


@pytest.mark.parametrize("S,prefix", [(300, 1040), (64, 4096), (2048, 64)])
def test_mixed_batches(ops, S, prefix):  # noqa: F811
    """Any share of the batch inside the prefix."""
    rng = np.random.default_rng(S)
    for inside in (0.02, 0.5, 0.98):
        lens = [int(rng.integers(0, prefix)) if rng.random() < inside else prefix + int(rng.integers(1, 40))
                for _ in range(S)]
        check(ops, problem(lens, [1] * S, 2, 1, 64, 16, prefix, seed=S))


def test_a_captured_step_while_the_prefix_fills(ops):  # noqa: F811
    """One graph, replayed while the lengths grow past the prefix's end."""
    prefix, S = 192, 5
    most = [prefix + 40 + s for s in range(S)]
    pb = problem(most, [1] * S, 8, 2, 128, 16, prefix, seed=4)
    clean = {k: pb[k].clone() for k in ("kc", "vc")}
    t = {k: pb[k].to(DEV) for k in ("q", "kc", "vc")}
    bt, table = torch.from_numpy(pb["bt"]).to(DEV), torch.from_numpy(pb["table"]).to(DEV)
    lens = torch.zeros(S, dtype=torch.int32, device=DEV)
    out = torch.empty_like(t["q"])
    ws = torch.empty(max(256, ops.prefix_workspace_bytes(S, S, 1, 300, prefix, 8, 2, 128, 16, torch.bfloat16)),
                     dtype=torch.uint8, device=DEV)

    def go():
        ops.paged_attention_decode_prefix(t["q"], t["kc"], t["vc"], table, bt, lens, pb["scale"],
                                          prefix_len=prefix, max_context_len=300, out=out, workspace=ws)
    go()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        go()
    for at in (0, 1, 100, 190, 191, 192, 193, 230, 3):
        now = [min(m, at + s) for s, m in enumerate(most)]
        pb.update(lens=now, kc=clean["kc"].clone(), vc=clean["vc"].clone())
        stale(pb, max(now))
        t["kc"].copy_(pb["kc"])
        t["vc"].copy_(pb["vc"])
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        check(ops, pb, out)
