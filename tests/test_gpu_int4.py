"""4-bit KV pages on the GPU against the oracle: codes, scales and offsets bit
for bit, attention within the tolerance of the other pools."""

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests._helpers import as_f64, check_attention, storage

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_115_gb300 import build
    build.build()
    from paged_kv_cache_115_gb300 import ops as o
    o.get_device_error()
    return o


def empty_pool(nb, K, H, D, rng):
    codes = torch.from_numpy(rng.integers(0, 256, (nb, K, H, D // 2)).astype(np.uint8))
    words = torch.from_numpy(rng.integers(-32768, 32768, (nb, H, K, 2)).astype(np.int16))
    return codes, words.view(torch.bfloat16)


def rows_like(T, H, D, dtype, rng):
    """Rows of different sizes and offsets, and special ones."""
    x = rng.standard_normal((T, H, D)) * 10.0 ** rng.integers(-3, 3, (T, H, 1)) \
        + rng.standard_normal((T, H, 1)) * 10.0 ** rng.integers(-3, 4, (T, H, 1))
    x = x.astype(np.float32)
    special = [np.zeros(D), np.full(D, -1.001), np.arange(D) % 16, np.full(D, -0.0),
               np.where(np.arange(D) == 3, np.nan, 1), np.where(np.arange(D) == D - 1, np.inf, 1),
               np.where(np.arange(D) == 0, -np.inf, 1), np.arange(D) * 1e-39, np.arange(D) * 3e-38,
               np.where(np.arange(D) % 2, 3.0e38, -3.0e38), np.where(np.arange(D) % 2, 1.7e38, 0),
               100 + np.arange(D) / D]
    flat = x.reshape(T * H, D)
    for i, s in enumerate(special[:T * H]):
        flat[(i * 7) % (T * H)] = s.astype(np.float32)
    return torch.from_numpy(x).to(dtype)


def same_pool(got_codes, got_scales, codes, scales):
    """Codes equal; scales and offsets equal as values (a zero's sign and a
    NaN's payload are free)."""
    assert np.array_equal(got_codes.cpu().numpy(), codes)
    g, w = storage(got_scales), scales
    nan = lambda a: (a & 0x7FFF) > 0x7F80
    same = (g == w) | (nan(g) & nan(w)) | (((g | w) & 0x7FFF) == 0)
    assert same.all()


SHAPES = [(1, 1, 64, 8), (1, 8, 128, 16), (3, 2, 128, 1), (61, 3, 64, 32), (257, 8, 128, 16),
          (5, 7, 128, 24), (1300, 8, 128, 16), (4099, 8, 64, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,K", SHAPES)
def test_write(ops, T, H, D, K, dtype):
    rng = np.random.default_rng(T * 100 + D + K)
    nb = -(-T // K) + 3
    kc, ks = empty_pool(nb, K, H, D, rng)
    vc, vs = empty_pool(nb, K, H, D, rng)
    k, v = rows_like(T, H, D, dtype, rng), rows_like(T, H, D, dtype, rng)
    slots = rng.permutation(nb * K)[:T].astype(np.int64)
    slots[T // 2::17] = -1
    want = Q.kv_write_int4(kc.numpy(), vc.numpy(), storage(ks), storage(vs), k.float().numpy(),
                           v.float().numpy(), slots)
    # cut out of one projection's output, on 16-byte boundaries and off them
    for lead, pad in ((0, 0), (8, 16), (1, 0), (0, 3)):
        wide = torch.zeros((T, lead + 2 * H * D + pad), dtype=dtype)
        wide[:, lead:lead + H * D] = k.reshape(T, -1)
        wide[:, lead + H * D:lead + 2 * H * D] = v.reshape(T, -1)
        wide = wide.to(DEV)
        gk = wide[:, lead:lead + H * D].view(T, H, D)
        gv = wide[:, lead + H * D:lead + 2 * H * D].view(T, H, D)
        d = [t.to(DEV) for t in (kc, vc, ks, vs)]
        ops.paged_kv_write_quant(gk, gv, torch.from_numpy(slots).to(DEV), d[0], d[1],
                                 ops.kv_quant("int4", k_token_scales=d[2], v_token_scales=d[3]))
        same_pool(d[0], d[2], want[0], want[2])
        same_pool(d[1], d[3], want[1], want[3])
    assert ops.get_device_error() == 0


def test_write_slots_out_of_range(ops):
    rng = np.random.default_rng(5)
    nb, K, H, D = 4, 8, 2, 64
    kc, ks = empty_pool(nb, K, H, D, rng)
    d = [t.to(DEV) for t in (kc, kc.clone(), ks, ks.clone())]
    k = torch.randn((3, H, D), device=DEV)
    for slot in (nb * K, -2, 2**40, -2**62):
        slots = torch.tensor([slot, -1, slot], device=DEV)
        ops.paged_kv_write_quant(k, k, slots, d[0], d[1],
                                 ops.kv_quant("int4", k_token_scales=d[2], v_token_scales=d[3]))
        assert ops.get_device_error() == 2
        assert torch.equal(d[0].cpu(), kc) and np.array_equal(storage(d[3]), storage(ks))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_by_positions(ops, dtype):
    rng = np.random.default_rng(6)
    T, H, D, K, nb = 37, 4, 128, 16, 60
    kc, ks = empty_pool(nb, K, H, D, rng)
    vc, vs = empty_pool(nb, K, H, D, rng)
    k, v = rows_like(T, H, D, dtype, rng), rows_like(T, H, D, dtype, rng)
    bt = rng.permutation(nb)[:T].reshape(T, 1).astype(np.int32)
    bt = np.concatenate([np.full((T, 1), -5, np.int32), bt], 1)
    pos = (K + np.arange(T) % K).astype(np.int32)
    pos[4], pos[5], pos[6], bt[7, 1] = -1, 0, 2 * K, nb                # skipped; the last three recorded
    slots = np.where((pos >= K) & (pos < 2 * K), bt[:, 1].astype(np.int64) * K + pos - K, -1)
    slots[7] = -1
    want = Q.kv_write_int4(kc.numpy(), vc.numpy(), storage(ks), storage(vs), k.float().numpy(),
                           v.float().numpy(), slots)
    d = [t.to(DEV) for t in (kc, vc, ks, vs)]
    out = torch.empty(T, dtype=torch.int64, device=DEV)
    ops.paged_kv_append_quant(k.to(DEV), v.to(DEV), torch.from_numpy(bt).to(DEV),
                              torch.from_numpy(pos).to(DEV), d[0], d[1],
                              ops.kv_quant("int4", k_token_scales=d[2], v_token_scales=d[3]), out)
    assert ops.get_device_error() in (1, 5)
    assert np.array_equal(out.cpu().numpy(), slots)
    same_pool(d[0], d[2], want[0], want[2])
    same_pool(d[1], d[3], want[1], want[3])


@pytest.mark.parametrize("fmt", ["fp8", "int8", "k16v8"])
def test_write_other_formats(ops, fmt):
    # at the slots that positions and tables give: the same pools
    rng = np.random.default_rng(7)
    T, H, D, K, nb = 19, 2, 128, 16, 30
    k, v = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
            for _ in range(2))
    bt = torch.from_numpy(rng.permutation(nb)[:T].reshape(T, 1).astype(np.int32)).to(DEV)
    pos = torch.arange(T, device=DEV, dtype=torch.int32) % K
    pos[3] = -1

    def pools():
        c = torch.zeros((nb, K, H, D), dtype=torch.uint8, device=DEV)
        kc = c.to(torch.bfloat16) if fmt == "k16v8" else c.clone()
        s = torch.zeros(nb * K, device=DEV)
        if fmt == "int8":
            qd = ops.kv_quant("int8", k_token_scales=s.clone(), v_token_scales=s.clone())
        else:
            qd = ops.kv_quant(fmt, 0.5, 0.25)
        return kc, c.clone(), qd
    a, b = pools(), pools()
    slots = torch.empty(T, dtype=torch.int64, device=DEV)
    ops.paged_kv_append_quant(k, v, bt, pos, a[0], a[1], a[2], slots)
    wide = torch.cat([k.reshape(T, -1), v.reshape(T, -1)], 1)
    ops.paged_kv_write_quant(wide[:, :H * D].view(T, H, D), wide[:, H * D:].view(T, H, D), slots, b[0],
                             b[1], b[2])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if fmt == "int8":
        for x, y in zip(a[2]._scale_tensors, b[2]._scale_tensors):
            assert torch.equal(x, y)
    ops.paged_kv_write_quant(k, v, torch.full((T,), nb * K, device=DEV), b[0], b[1], b[2])
    assert ops.get_device_error() == 2
    assert torch.equal(a[0], b[0])


def test_block_copy(ops):
    rng = np.random.default_rng(8)
    nb, K, H, D = 9, 16, 3, 64
    kc, ks = empty_pool(nb, K, H, D, rng)
    vc, vs = empty_pool(nb, K, H, D, rng)
    d = [t.to(DEV) for t in (kc, vc, ks, vs)]
    pairs = torch.tensor([[0, 5], [3, 1]], device=DEV)
    ops.kv_block_copy_quant(d[0], d[1], pairs, ops.kv_quant("int4", k_token_scales=d[2], v_token_scales=d[3]))
    for got, t in zip(d, (kc, vc, ks, vs)):
        t = t.view(torch.int16) if t.dtype == torch.bfloat16 else t.clone()
        t[5], t[1] = t[0], t[3]
        got = got.view(torch.int16) if got.dtype == torch.bfloat16 else got
        assert torch.equal(got.cpu(), t)


# ---------------------------------------------------------------------------

def make(lens, H_q, H_kv, D, K, dtype, seed, spread=1.0, shift=0.0, share=0, group=1):
    """A batch over a pool whose slots without a token hold NaN scales; the rows of
    a group of ``group`` sequences list the same first ``share`` blocks."""
    rng = np.random.default_rng(seed)
    S = len(lens)
    nblk = [-(-L // K) for L in lens]
    nb = sum(nblk) + 3
    order = rng.permutation(nb)
    bt = rng.integers(-2**31, 2**31, (S, max(nblk) + 2)).astype(np.int32)
    used, at = np.zeros((nb, K), bool), 0
    for s in range(S):
        bt[s, :nblk[s]] = order[at:at + nblk[s]]
        at += nblk[s]
        if s % group:
            n = min(share, nblk[s], nblk[s - s % group])
            bt[s, :n] = bt[s - s % group, :n]
        t = np.arange(lens[s])
        used[bt[s, t // K], t % K] = True
    pools = []
    for _ in range(2):
        x = rng.standard_normal((nb, K, H_kv, D)) * spread + shift * rng.standard_normal((1, 1, H_kv, D))
        c, s_, z = Q.int4_quantize(x.astype(np.float32))
        codes = np.where(used[:, :, None, None], Q.int4_pack(c), 0xA5).astype(np.uint8)
        scales = np.where(used[:, :, None, None], np.stack([s_, z], -1), 0x7FC0).astype(np.uint16)
        pools += [codes, np.ascontiguousarray(scales.transpose(0, 2, 1, 3))]
    q = torch.from_numpy(rng.standard_normal((S, H_q, D)).astype(np.float32)).to(dtype)
    return q, pools[0], pools[2], pools[1], pools[3], bt, np.array(lens, np.int32)


def on_gpu(ops, c):
    q, kc, vc, ks, vs, bt, lens = c
    words = [torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).to(DEV) for w in (ks, vs)]
    return (q.to(DEV), torch.from_numpy(kc).to(DEV), torch.from_numpy(vc).to(DEV),
            torch.from_numpy(bt).to(DEV), torch.from_numpy(lens).to(DEV),
            ops.kv_quant("int4", k_token_scales=words[0], v_token_scales=words[1]))


def check(ops, c, scale, **kw):
    q, kc, vc, ks, vs, bt, lens = c
    g = on_gpu(ops, c)
    out = ops.paged_attention_decode_quant(*g[:5], scale, g[5], max_context_len=int(max(lens.max(), 1)), **kw)
    assert ops.get_device_error() == 0
    dt = "bf16" if q.dtype == torch.bfloat16 else "f32"
    ref = Q.paged_attention_decode_int4(storage(q), kc, vc, ks, vs, bt, lens, scale, dt)
    check_attention(as_f64(out), ref, dt)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H_q,H_kv,D,K", [(4, 2, 64, 8), (8, 8, 128, 16), (16, 2, 128, 24),
                                          (5, 1, 128, 5), (32, 2, 64, 32)])
@pytest.mark.parametrize("lens", [[1], [0, 17, 1, 33, 600], [1025, 0, 0, 16]])
def test_attention(ops, lens, H_q, H_kv, D, K, dtype):
    check(ops, make(lens, H_q, H_kv, D, K, dtype, seed=sum(lens) + D), D ** -0.5, kernel=2)
    check(ops, make(lens, H_q, H_kv, D, K, dtype, seed=sum(lens) + K), D ** -0.5)


def test_attention_bad_block_reads_zeros(ops):
    c = make([40, 40], 8, 2, 128, 16, torch.bfloat16, seed=3)
    q, kc, vc, ks, vs, bt, lens = c
    bt[1, 1] = kc.shape[0]
    g = on_gpu(ops, c)
    for kernel in (0, 2):
        out = ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=40, kernel=kernel)
        assert ops.get_device_error() == 1
        # the block as 16 rows of zeros
        kz, vz, ksz, vsz = kc.copy(), vc.copy(), ks.copy(), vs.copy()
        free = next(b for b in range(kc.shape[0]) if b not in set(bt[:, :3].flatten().tolist()))
        kz[free], vz[free], ksz[free], vsz[free] = 0, 0, 0, 0
        bz = bt.copy()
        bz[1, 1] = free
        ref = Q.paged_attention_decode_int4(storage(q), kz, vz, ksz, vsz, bz, lens, 0.1, "bf16")
        check_attention(as_f64(out), ref, "bf16")


def test_attention_reads_nan_of_rows_that_were_not_finite(ops):
    c = make([20, 20], 4, 1, 128, 16, torch.bfloat16, seed=4)
    q, kc, vc, ks, vs, bt, lens = c
    vs[bt[0, 0], 0, 3] = 0x7FFF
    g = on_gpu(ops, c)
    out = ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=20).cpu()
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


# the tensor-core kernel: head counts that give 8, 4, 2 and 1 heads a CTA, several
# groups of KV heads, 8-token blocks, long tables, splits
TC_LENS = [[1], [31, 32, 33], [0, 17, 1, 0, 600, 64, 0], [3000, 5, 1025]]


@pytest.mark.parametrize("lens", TC_LENS)
@pytest.mark.parametrize("H_q,H_kv,K", [(32, 8, 16), (8, 8, 8), (16, 16, 32), (28, 4, 16), (12, 12, 8), (16, 2, 8),
                                        (2, 2, 64), (7, 1, 16), (8, 1, 8), (24, 3, 48), (40, 10, 16)])
def test_attention_tensor_cores(ops, lens, H_q, H_kv, K):
    c = make(lens, H_q, H_kv, 128, K, torch.bfloat16, seed=sum(lens) + H_q + K)
    a = check(ops, c, 128 ** -0.5, kernel=1)
    b = check(ops, c, 128 ** -0.5, kernel=1, num_splits=3)
    assert (a.float() - b.float()).abs().max() < 4e-3
    assert torch.equal(a, check(ops, c, 128 ** -0.5, kernel=1))


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("spread,shift,scale", [(1e-4, 0, 30.0), (1e4, 0, 1e-6), (0.1, 30.0, 1e-3), (1.0, 0.0, 2.0),
                                                (3e-30, 0, 0.0), (1.0, 3.0, -0.1)])
def test_attention_sizes_of_values(ops, spread, shift, scale, kernel):
    # V from far below to far above 1, offsets far from 0, sharp and flat softmax; the
    # tolerance scales with the largest output
    c = make([500, 77], 16, 4, 128, 16, torch.bfloat16, seed=11, spread=spread, shift=shift)
    q, kc, vc, ks, vs, bt, lens = c
    g = on_gpu(ops, c)
    out = as_f64(ops.paged_attention_decode_quant(*g[:5], scale, g[5], max_context_len=500, kernel=kernel))
    ref = Q.paged_attention_decode_int4(storage(q), kc, vc, ks, vs, bt, lens, scale, "bf16")
    top = np.abs(ref).max()
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= 2e-3 * top + 1e-2 * np.abs(ref)).all()


def test_attention_scale_jumps(ops):
    # V scales that grow and shrink by powers of ten along a sequence
    c = make([700], 8, 2, 128, 16, torch.bfloat16, seed=12)
    q, kc, vc, ks, vs, bt, lens = c
    rng = np.random.default_rng(0)
    for t in range(700):
        f = np.float32(10.0 ** rng.integers(-6, 3))
        for h in range(2):
            w = (vs[bt[0, t // 16], h, t % 16].astype(np.uint32) << np.uint32(16)).view(np.float32) * f
            vs[bt[0, t // 16], h, t % 16] = Q.bf16_encode(w)
    g = on_gpu(ops, c)
    for kernel in (1, 2):
        out = as_f64(ops.paged_attention_decode_quant(*g[:5], 0.1, g[5], max_context_len=700, kernel=kernel))
        ref = Q.paged_attention_decode_int4(storage(q), kc, vc, ks, vs, bt, lens, 0.1, "bf16")
        assert (np.abs(out - ref) <= 2e-3 * np.abs(ref).max() + 1e-2 * np.abs(ref)).all()


@pytest.mark.parametrize("H_q,H_kv,K,group", [(32, 8, 16, 4), (16, 8, 16, 3), (8, 8, 8, 16), (28, 4, 32, 2),
                                              (8, 1, 16, 5), (6, 2, 8, 5), (16, 16, 16, 8)])
def test_attention_shared_prefix(ops, H_q, H_kv, K, group):
    rng = np.random.default_rng(H_q + K)
    lens = [int(x) for x in rng.integers(1, 400, 3 * group + 1)]
    lens[1], lens[-1] = 0, 900
    for share in (0, 1, 7, 30):
        c = make(lens, H_q, H_kv, 128, K, torch.bfloat16, seed=share, share=share, group=group)
        check(ops, c, 128 ** -0.5, share_prefix=True)
        check(ops, c, 128 ** -0.5, share_prefix=True, kernel=1, num_splits=5)
