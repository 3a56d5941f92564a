"""GPU parity of norm + rotation + append against oracle/step.py (float64).

Tolerances.  Between load and store everything is float32: the mean of
squares of D values takes D/32 sums in a lane and 5 in the warp, the
reciprocal root (2 ulp) halves its relative error, two products and the
rotation (two products, one sum) follow.  For D <= 512 that is at most
(512/32 + 5 + 3) / 2 + 4 + 2 + 3 < 24 steps of 2^-24, relative to |a| + |b| of
the rotated pair.  The store rounds once: half a step of the type, relative to
the value (e4m3: also half of its smallest step 2^-9).
"""

import numpy as np
import pytest
import torch

from oracle import quant as OQ
from oracle import step as O
from tests._helpers import as_f64, storage

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32_STEPS = 24 * 2.0**-24


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def problem(T, H, J, D, K, rot, dtype, seed=0, far=300, gap=0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    width = (H + 2 * J) * D + gap
    qkv = torch.randn((T, width), generator=g).to(dtype)
    nb = -(-T // K) + 3
    slots = rng.permutation(nb * K)[:T].astype(np.int64)
    pos = rng.integers(0, far, T).astype(np.int32)
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    ang = np.arange(far)[:, None] * inv[None]
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = (1 + 0.2 * torch.randn((2, D), generator=g)).to(dtype)
    return dict(T=T, H=H, J=J, D=D, K=K, rot=rot, nb=nb, qkv=qkv, slots=slots, pos=pos,
                table=table, wq=w[0], wk=w[1], eps=1e-6)


def views(pb, qkv):
    H, J, D, T = pb["H"], pb["J"], pb["D"], pb["T"]
    a, b = H * D, (H + J) * D
    return (qkv[:, :a].unflatten(1, (H, D)), qkv[:, a:b].unflatten(1, (J, D)),
            qkv[:, b:b + J * D].unflatten(1, (J, D)))


def want_rows(pb, x, w, interleaved):
    """(rows in float64, |a| + |b| of each value's pair)"""
    T, H, D = x.shape
    rows = np.empty((T, H, D))
    mag = np.empty((T, H, D))
    half = pb["rot"] // 2
    for t in range(T):
        for h in range(H):
            y = O.norm_rope(x[t, h], w, pb["eps"], 0, np.concatenate([np.ones((1, half)), np.zeros((1, half))], 1), interleaved)
            rows[t, h] = O.norm_rope(x[t, h], w, pb["eps"], int(pb["pos"][t]), pb["table"], interleaved)
            m = np.abs(y)
            mag[t, h] = m
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                mag[t, h, a] = mag[t, h, b] = m[a] + m[b]
    return rows, mag


def near(got, ref, mag, dtype, what):
    half = torch.finfo(dtype).eps / 2
    err = np.abs(got - ref)
    tol = half * np.abs(ref) + (1 + half) * F32_STEPS * mag
    assert np.all(err <= tol), (what, float((err - tol).max()))


def run(ops, pb, dtype, norm, interleaved, in_place=False):
    qkv = pb["qkv"].to(DEV)
    q, k, v = views(pb, qkv)
    nan = float("nan")
    kc = torch.full((pb["nb"], pb["K"], pb["J"], pb["D"]), nan, dtype=dtype, device=DEV)
    vc = kc.clone()
    out = ops.paged_qk_norm_rope_append(
        q, k, v, torch.from_numpy(pb["pos"]).to(DEV), torch.from_numpy(pb["slots"]).to(DEV), kc,
        vc, torch.from_numpy(pb["table"]).to(DEV), q_weight=pb["wq"].to(DEV) if norm else None,
        k_weight=pb["wk"].to(DEV) if norm else None, eps=pb["eps"], interleaved=interleaved,
        q_out=q if in_place else None)
    return out, kc, vc, qkv


def check(ops, pb, dtype, norm, interleaved, in_place=False):
    out, kc, vc, qkv = run(ops, pb, dtype, norm, interleaved, in_place)
    assert ops.get_device_error() == 0
    q, k, v = views(pb, pb["qkv"])
    J, D = pb["J"], pb["D"]
    ref, mag = want_rows(pb, as_f64(q), as_f64(pb["wq"]) if norm else None, interleaved)
    near(as_f64(out), ref, mag, dtype, "q")
    ref, mag = want_rows(pb, as_f64(k), as_f64(pb["wk"]) if norm else None, interleaved)
    flat = kc.view(-1, J, D)
    near(as_f64(flat[torch.from_numpy(pb["slots"]).to(DEV)]), ref, mag, dtype, "k")
    fv = storage(vc).reshape(-1, J, D)
    assert np.array_equal(fv[pb["slots"]], storage(v))                  # V bit for bit
    rest = np.setdiff1d(np.arange(pb["nb"] * pb["K"]), pb["slots"])     # other slots untouched
    assert np.isnan(as_f64(flat)[rest]).all() and np.isnan(as_f64(vc.view(-1, J, D))[rest]).all()
    # the projection's output is untouched, apart from q in place
    skip = pb["H"] * D if in_place else 0
    assert torch.equal(qkv[:, skip:].cpu(), pb["qkv"][:, skip:])


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (256, 256), (80, 32), (96, 96),
                                   (2, 2), (126, 10), (512, 512), (64, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(ops, D, rot, dtype, interleaved):
    pb = problem(5, 6, 2, D, 4, rot, dtype, seed=D + rot)
    check(ops, pb, dtype, True, interleaved)
    check(ops, pb, dtype, False, interleaved)


@pytest.mark.parametrize("H,J", [(1, 1), (3, 3), (32, 8), (64, 8), (7, 1), (16, 16)])
@pytest.mark.parametrize("T", [1, 2, 33])
def test_heads_and_tokens(ops, H, J, T):
    pb = problem(T, H, J, 128, 16, 128, torch.bfloat16, seed=H + T)
    check(ops, pb, torch.bfloat16, True, False)
    check(ops, pb, torch.bfloat16, T != 2, False, in_place=True)


@pytest.mark.parametrize("gap", [1, 2, 4, 8, 129])
def test_strides(ops, gap):
    """Rows cut out of a wider projection: every alignment of a row's start."""
    for dtype in (torch.bfloat16, torch.float32):
        check(ops, problem(7, 4, 2, 64, 8, 64, dtype, seed=gap, gap=gap), dtype, True, False)
        check(ops, problem(7, 4, 2, 64, 8, 32, dtype, seed=gap, gap=gap), dtype, True, True)


def test_more_tokens_than_one_wave(ops):
    """Thousands of tokens: every row against a vectorised float64 form."""
    T, H, J, D = 5000, 32, 8, 128
    pb = problem(T, H, J, D, 16, D, torch.bfloat16, seed=3)
    out, kc, vc, _ = run(ops, pb, torch.bfloat16, True, False)
    assert ops.get_device_error() == 0
    q, k, v = views(pb, pb["qkv"])
    cs = torch.from_numpy(pb["table"])[torch.from_numpy(pb["pos"]).long()].double()[:, None]
    for x, w, got in ((q, pb["wq"], out.cpu()),
                      (k, pb["wk"], kc.view(-1, J, D).cpu()[torch.from_numpy(pb["slots"])])):
        y = x.double()
        y = y / (y.pow(2).mean(-1, keepdim=True) + pb["eps"]).sqrt() * w.double()
        a, b = y[..., :64], y[..., 64:]
        ref = torch.cat([a * cs[..., :64] - b * cs[..., 64:], b * cs[..., :64] + a * cs[..., 64:]], -1)
        mag = (a.abs() + b.abs()).repeat(1, 1, 2)
        near(got.double().numpy(), ref.numpy(), mag.numpy(), torch.bfloat16, "rows")
    assert torch.equal(vc.view(-1, J, D).cpu()[torch.from_numpy(pb["slots"])], v)


@pytest.mark.parametrize("fmt", ["fp8", "int8", "k16v8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,J", [(128, 16, 8), (64, 4, 1), (96, 6, 2)])
def test_quantized_pools(ops, fmt, dtype, D, H, J):
    pb = problem(19, H, J, D, 8, D, dtype, seed=D)
    nb, K, T = pb["nb"], pb["K"], pb["T"]
    qkv = pb["qkv"].to(DEV)
    q, k, v = views(pb, qkv)
    shape = (nb, K, J, D)
    kc = torch.full(shape, 99, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    ks, vs = 0.03125, 0.015625
    if fmt == "k16v8":
        kc = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
    kts = torch.full((nb * K,), 5.0, device=DEV)
    vts = kts.clone()
    quant = ops.kv_quant(fmt, ks, vs, kts, vts)
    out = ops.paged_qk_norm_rope_append(
        q, k, v, torch.from_numpy(pb["pos"]).to(DEV), torch.from_numpy(pb["slots"]).to(DEV), kc,
        vc, torch.from_numpy(pb["table"]).to(DEV), pb["wq"].to(DEV), pb["wk"].to(DEV),
        eps=pb["eps"], quant=quant)
    assert ops.get_device_error() == 0
    qr, kr, vr = views(pb, pb["qkv"])
    ref, mag = want_rows(pb, as_f64(qr), as_f64(pb["wq"]), False)
    near(as_f64(out), ref, mag, dtype, "q")
    ref, mag = want_rows(pb, as_f64(kr), as_f64(pb["wk"]), False)
    sl = pb["slots"]
    v32 = as_f64(vr).astype(np.float32)
    got_k = kc.view(-1, J, D).cpu()[torch.from_numpy(sl)]
    got_v = vc.view(-1, J, D).cpu()[torch.from_numpy(sl)].numpy()
    if fmt == "int8":
        amax = np.abs(ref).reshape(T, -1).max(1)
        worst = F32_STEPS * mag.reshape(T, -1).max(1)
        sc = as_f64(kts)[sl]
        assert np.all(np.abs(sc - amax / 127) <= (worst + amax * 2.0**-23) / 127)
        val = got_k.view(torch.int8).double().numpy() * sc[:, None, None]
        # half a step of the code, the row's float32 error, the quotient's rounding
        tol = 0.5 * sc[:, None, None] * (1 + 2.0**-15) + F32_STEPS * mag + (worst + amax * 2.0**-22)[:, None, None]
        assert np.all(np.abs(val - ref) <= tol)
        for t in range(T):
            codes, s = OQ.int8_token_quantize(v32[t].reshape(-1))
            assert np.array_equal(got_v[t].view(np.int8).reshape(-1), codes)
            assert np.float32(s) == vts.cpu().numpy()[sl[t]]
        assert (kts.cpu().numpy()[np.setdiff1d(np.arange(nb * K), sl)] == 5.0).all()
    else:
        assert np.array_equal(got_v, OQ.e4m3_encode(v32 / np.float32(vs)))
        if fmt == "k16v8":
            near(as_f64(got_k), ref, mag, torch.bfloat16, "k")
        else:
            val = OQ.e4m3_decode(got_k.numpy())
            r = np.clip(ref / ks, -448, 448)
            tol = 2.0**-4 * np.abs(r) + 2.0**-10 + (1 + 2.0**-4) * (F32_STEPS * mag / ks + 2.0**-24 * np.abs(r))
            assert np.all(np.abs(val - r) <= tol)
    rest = np.setdiff1d(np.arange(nb * K), sl)
    assert (vc.view(-1, J, D).cpu().numpy()[rest] == 99).all()


def test_padding_and_bad_places(ops):
    """Negative positions skip the token, slot -1 skips the pages, what is out
    of range is skipped and recorded."""
    pb = problem(6, 4, 2, 64, 4, 64, torch.bfloat16, seed=1)
    pb["pos"][1] = -1
    pb["slots"][3] = -1
    base = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    args = lambda: (*views(pb, pb["qkv"].to(DEV)), torch.from_numpy(pb["pos"]).to(DEV),  # noqa: E731
                    torch.from_numpy(pb["slots"]).to(DEV))
    table = torch.from_numpy(pb["table"]).to(DEV)

    def go():
        kc = torch.full((pb["nb"], 4, 2, 64), 2.0, dtype=torch.bfloat16, device=DEV)
        vc = kc.clone()
        out = ops.paged_qk_norm_rope_append(*args(), kc, vc, table, pb["wq"].to(DEV),
                                            pb["wk"].to(DEV), q_out=base.clone())
        return out.cpu(), kc.view(-1, 2, 64).cpu(), vc.view(-1, 2, 64).cpu()
    out, kc, vc = go()
    assert ops.get_device_error() == 0
    assert (out[1] == 3.0).all() and not (out[3] == 3.0).any()
    written = [int(pb["slots"][t]) for t in (0, 2, 4, 5)]
    for c in (kc, vc):
        mask = torch.ones(c.shape[0], dtype=torch.bool)
        mask[written] = False
        assert (c[mask] == 2.0).all() and not (c[~mask] == 2.0).all(-1).any()
    pb["pos"][0] = 300
    out2, kc2, _ = go()
    assert ops.get_device_error() == 5 and (out2[0] == 3.0).all()
    assert (kc2[written[0]] == 2.0).all() and torch.equal(out2[2:], out[2:])
    pb["pos"][0] = 5
    pb["slots"][2] = pb["nb"] * 4
    out3, kc3, _ = go()
    assert ops.get_device_error() == 2 and torch.equal(out3[2], out[2])
    assert (kc3[written[1]] == 2.0).all()


def test_zero_rows_and_infinities(ops):
    """A zero row stays zero; an infinite value makes its own head NaN and no
    other."""
    pb = problem(3, 2, 1, 128, 4, 128, torch.bfloat16, seed=2)
    pb["qkv"][0, :128] = 0
    pb["qkv"][1, 5] = float("inf")
    out, kc, vc, _ = run(ops, pb, torch.bfloat16, True, False)
    o = as_f64(out)
    assert (o[0, 0] == 0).all() and np.isnan(o[1, 0]).any()
    assert np.isfinite(o[1, 1]).all() and np.isfinite(o[2]).all() and np.isfinite(o[0]).all()


def test_refused_arguments(ops):
    pb = problem(4, 4, 2, 64, 4, 64, torch.bfloat16)
    q, k, v = views(pb, pb["qkv"].to(DEV))
    pos, sl = torch.from_numpy(pb["pos"]).to(DEV), torch.from_numpy(pb["slots"]).to(DEV)
    kc = torch.zeros((pb["nb"], 4, 2, 64), dtype=torch.bfloat16, device=DEV)
    t = torch.from_numpy(pb["table"]).to(DEV)
    f = ops.paged_qk_norm_rope_append
    with pytest.raises(ValueError):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, pos, sl, kc, kc, t)
    with pytest.raises(TypeError):
        f(q.float(), k, v, pos, sl, kc, kc, t)
    with pytest.raises(TypeError):
        f(q, k, v, pos.long(), sl, kc, kc, t)
    with pytest.raises(ValueError):
        f(q, k, v, pos[:3], sl, kc, kc, t)
    with pytest.raises(ops.PagedKVError):
        f(q, k, v, pos, sl, kc, kc, t[:, :63].contiguous())
    with pytest.raises(ops.PagedKVError):
        f(q, k, v, pos, sl, kc, kc, torch.zeros((4, 66), device=DEV))
    with pytest.raises(ValueError):
        f(q, k, v, pos, sl.cpu(), kc, kc, t)
    with pytest.raises(TypeError):
        f(q, k, v, pos, sl, kc, kc, t.double())
    codes = torch.zeros(kc.shape, dtype=torch.uint8, device=DEV)
    with pytest.raises(TypeError):
        f(q, k, v, pos, sl, kc, codes, t, quant=ops.kv_quant("fp8"))
    with pytest.raises(TypeError):
        f(q, k, v, pos, sl, codes, codes, t, quant=ops.kv_quant("k16v8"))
    with pytest.raises(TypeError):
        f(q, k, v, pos, sl, kc, kc, t, quant=ops.kv_quant("k16v8"))
    with pytest.raises(ValueError):
        f(q, k, v, pos, sl, codes, codes[:-1], t, quant=ops.kv_quant("fp8"))
    few = torch.zeros(3, device=DEV)
    with pytest.raises(ValueError):
        f(q, k, v, pos, sl, codes, codes, t, quant=ops.kv_quant("int8", 1.0, 1.0, few, few))
