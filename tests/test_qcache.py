"""The 4-bit cache (fa_qcache_*) against its definition in 64 bits.

Bounds.  Reading rounds a stored value times the tensor's scale once (2^-8).
Attention works on the stored values exactly; its errors are
  - the score: products of fp16 operands are exact, their fp32 sums over d
    channels are off by at most 16 roundings of 2^-23 of sum |q k| (8 steps of
    16 channels, each with one sum inside and one onto the accumulator), and
    the scaling and the exponential's argument by 2^-22 of |score|:
    delta = 2^-18 * big (big the largest scale * sum |q k| >= |score|), plus
    the exponential's 2^-21: a probability is off by that share of itself;
  - a probability's rounding to fp16: 2^-11;
  - the result's rounding to bf16: 2^-8 of it.
So |o - o64| <= 2^-8 |o| + (2^-11 + 2 delta + 2^-20) sum p |v|, and
|lse - lse64| <= delta + 2^-21 (|lse| + 1).
"""
import math

import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref

gpu = pytest.mark.gpu


def rand(shape, seed, mult=1.0):
    return (torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)) * mult).to(torch.bfloat16)


def dev(*ts):
    return tuple(t.cuda() for t in ts)


def check_attention(o, lse, q, cache, causal, scale, what="", k_scale=1.0, v_scale=1.0):
    pool, table, lens = cache
    ks, vs = ref.unpack(pool, table, lens, q.shape[-1], k_scale, v_scale)
    o64, lse64, mag, big = ref.attention(q, ks, vs, causal, scale)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    delta = 2.0 ** -18 * big
    err = np.abs(o - o64)
    assert (err <= 2.0 ** -8 * np.abs(o64) + (2.0 ** -11 + 2.0 ** -20 + 2 * delta[..., None]) * mag).all(), \
        f"{what}: o off by {err.max():.3e}"
    seen = lse64 > -np.inf
    assert np.array_equal(lse > -np.inf, seen), what
    err = np.abs(lse - lse64)[seen]
    bound = (delta + 2.0 ** -21 * (np.abs(np.where(seen, lse64, 0)) + 1))[seen]
    assert (err <= bound).all(), f"{what}: lse off by {err.max():.3e}"


# --------------------------------------------------------------- the definition

def test_reference_rounding_pins():
    """The helper itself, on the CPU: codes of the grid and of its halves, the scale's clamp and its flush."""
    x = np.zeros((1, 64))
    x[0, :16] = [6, -6, 4, 3, 2, 1.5, 1, 0.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25]
    code, byte = ref.quantise(x)
    assert ref.E4M3[byte[0, 0]] == 1.0
    assert ref.value(code, byte)[0, :16].tolist() == [6, -6, 4, 3, 2, 1.5, 1, 0.5, 0, 1, 1, 2, 2, 4, 4, 0]
    assert ref.E4M3[126] == 448 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[1] == 2.0 ** -9
    code, byte = ref.quantise(np.full((1, 64), 1e6))
    assert (ref.value(code, byte) == 2688).all()
    code, byte = ref.quantise(np.full((1, 64), 1e-4))
    assert (ref.value(code, byte) == 0).all()
    pool, table, lens = ref.make_cache([70, 0, 1], 2, 40, seed=1)
    ks, vs = ref.unpack(pool, table, lens, 40)
    assert [k.shape for k in ks] == [(2, 70, 40), (2, 0, 40), (2, 1, 40)] and np.isfinite(np.concatenate([v.ravel() for v in vs])).all()
    kc, kscale, vc, vscale = ref.places(64)
    assert len({*kc.ravel(), *kscale.ravel(), *vc.ravel(), *vscale.ravel()}) == 72 * 64  # every byte has its use


# -------------------------------------------------------------- append and read

def run_append(k, v, lens, d, seed=0, max_pages=None, k_scale=1.0, v_scale=1.0, table=None, views=False):
    """Appends into a junk-filled pool; checks that only the new keys' places changed.  Returns the cache."""
    B, Hkv, N, _ = k.shape
    rng = np.random.default_rng(seed)
    D = ref.stored_channels(d)
    need = max(1, max(-(-int(n) // 64) for n in lens)) if max_pages is None else max_pages
    count = B * need + 2
    if table is None:
        table = torch.from_numpy(rng.permutation(count)[:B * need].astype(np.int32)).reshape(B, need)
    pool = torch.from_numpy(rng.integers(0, 256, (count, Hkv, 72 * D), dtype=np.uint8))
    lens = torch.tensor(lens, dtype=torch.int32)
    kd, vd, pd, td, ld = dev(k, v, pool, table, lens)
    if views:  # (B, N, 2, Hkv, d) seen as k and v
        both = torch.stack([kd.transpose(1, 2), vd.transpose(1, 2)], 2).contiguous()
        kd, vd = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    fa.qcache_append(kd, vd, pd, td, ld, k_scale, v_scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    got = pd.cpu()
    # Bits that belong to a new key.
    mine = np.zeros(pool.shape, np.uint8)
    kc, ks, vc, vs = ref.places(D)
    for b, n in enumerate(lens.tolist()):
        for x in range(max(0, n - N), n):
            page, r = int(table[b, x // 64]), x % 64
            mine[page][:, kc[r]] = mine[page][:, ks[r]] = mine[page][:, vs[r]] = 255
            mine[page][:, vc[r]] |= 15 if r % 2 == 0 else 240
    assert np.array_equal(got.numpy() & ~mine, pool.numpy() & ~mine), "bytes of other keys changed"
    return got, table, lens


def expect_rows(x, n, N):
    """The rows of x (Hkv, N, d) that are keys, with their positions' order: the newest min(n, N)."""
    return x[:, max(0, N - n):]


@gpu
@pytest.mark.parametrize("d", [64, 128, 8, 40, 72, 120])
@pytest.mark.parametrize("N, lens", [(1, [1, 2, 64, 65, 0]), (5, [5, 3, 66, 129]), (64, [64, 100]), (131, [131, 130, 200, 1])])
def test_append_rounds_by_the_definition(d, N, lens):
    B, Hkv = len(lens), 3
    k, v = rand((B, Hkv, N, d), d + N, 2.0), rand((B, Hkv, N, d), d + N + 1, 0.5)
    cache = run_append(k, v, lens, d, seed=N)
    ks, vs = ref.unpack(*cache, d)
    for b, n in enumerate(lens):
        m = min(n, N)
        for got, x in ((ks[b], k), (vs[b], v)):
            code, byte = ref.quantise(expect_rows(x[b].double().numpy(), n, N))
            assert np.array_equal(got[:, n - m:], ref.value(code, byte)[..., :d])


@gpu
def test_append_meets_halves_clamps_and_extremes():
    """Every block has an exact half way, plus blocks of one large entry, tiny ones, zeros and non-finite ones."""
    d = 128
    x = torch.zeros((1, 1, 40, d))
    g = torch.Generator("cpu").manual_seed(3)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, -2.5, -5.0])
    for r in range(20):
        s = 2.0 ** (r - 8) * (1 + (r % 8) / 8)  # exactly an e4m3 scale
        x[0, 0, r] = mids[torch.randint(0, 10, (d,), generator=g)] * s
        x[0, 0, r, ::16] = 6 * s
    x[0, 0, 20] = torch.randn(d, generator=g) * 1e4
    x[0, 0, 21] = torch.randn(d, generator=g) * 1e-3
    x[0, 0, 22, 3] = 3e38
    x[0, 0, 23, 3], x[0, 0, 23, 4] = float("inf"), float("-inf")
    x[0, 0, 24, 3], x[0, 0, 24, 40] = float("nan"), 5.0
    x[0, 0, 25] = 6 * 2.0 ** -10  # the scale's own half way: to even, 0
    x[0, 0, 26:] = torch.randn((14, d), generator=g) * torch.exp(3 * torch.randn((14, d), generator=g))
    x = x.to(torch.bfloat16)
    cache = run_append(x, x.flip(2), [40], d)
    ks, vs = ref.unpack(*cache, d)
    for got, y in ((ks[0], x[0]), (vs[0], x[0].flip(1))):
        y = y.double().numpy()
        want = ref.value(*ref.quantise(y))
        assert np.isfinite(got).all() and np.array_equal(got, want)


@gpu
@pytest.mark.parametrize("k_scale, v_scale", [(0.013, 7.3), (2.0 ** -5, 3.0)])
def test_append_and_read_with_tensor_scales(k_scale, v_scale):
    """With a scale that is no power of two a quotient can lie within fp32's rounding of a half: each code is
    the nearest up to 2^-13 of the block's scale, and the block's scale is the nearest e4m3 or its neighbour
    at a half."""
    B, Hkv, N, d = 2, 2, 90, 96
    k, v = rand((B, Hkv, N, d), 1, k_scale * 3), rand((B, Hkv, N, d), 2, v_scale * 3)
    pool, table, lens = run_append(k, v, [90, 100], d, k_scale=k_scale, v_scale=v_scale)
    kr, vr = fa.qcache_read(*dev(pool, table, lens), N, d, newest=True, k_scale=k_scale, v_scale=v_scale)
    ks, vs = ref.unpack(pool, table, lens, d, k_scale, v_scale)
    for b, n in enumerate(lens.tolist()):
        for x, stored, read, scale in ((k, ks, kr, k_scale), (v, vs, vr, v_scale)):
            rows, got = x[b].double().numpy(), stored[b][:, n - N:]
            want = ref.value(*ref.quantise(rows, scale), scale)[..., :d]
            top = np.abs(np.pad(rows, ((0, 0), (0, 0), (0, 32))).reshape(Hkv, N, 8, 16)).max(-1).repeat(16, -1)[..., :d]
            err, best = np.abs(rows - got), np.abs(rows - want)
            assert (err <= best + 2.0 ** -13 * top).mean() > 0.999 and (err <= 0.35 * top).all()
            back = read[b].double().cpu().numpy()
            assert (np.abs(back - got) <= 2.0 ** -8 * np.abs(got)).all()


@gpu
def test_append_takes_views_and_leaves_the_neighbours():
    """k and v as strided views; one key at a time gives the same bytes as all at once."""
    B, Hkv, N, d = 2, 2, 70, 64
    k, v = rand((B, Hkv, N, d), 3), rand((B, Hkv, N, d), 4)
    a = run_append(k, v, [70, 80], d, seed=5, views=True)
    b = run_append(k, v, [70, 80], d, seed=5)
    assert torch.equal(a[0], b[0])
    rng = np.random.default_rng(5)
    rng.permutation(len(a[0]))
    pool = torch.from_numpy(rng.integers(0, 256, a[0].shape, dtype=np.uint8)).cuda()
    lens = torch.tensor([0, 10], dtype=torch.int32).cuda()
    table = a[1].cuda()
    for i in range(N):
        lens += 1
        fa.qcache_append(k[:, :, i:i + 1].contiguous().cuda(), v[:, :, i:i + 1].contiguous().cuda(), pool, table, lens)
    assert torch.equal(pool.cpu(), a[0])


@gpu
@pytest.mark.parametrize("newest", [False, True])
@pytest.mark.parametrize("d", [64, 128, 24, 88])
def test_read(newest, d):
    lens, n = [0, 1, 63, 64, 65, 200], 66
    pool, table, lens_t = ref.make_cache(lens, 2, d, seed=d)
    k, v = fa.qcache_read(*dev(pool, table, lens_t), n, d, newest=newest)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    ks, vs = ref.unpack(pool, table, lens_t, d)
    for b, m in enumerate(lens):
        for got, x in ((k, ks), (v, vs)):
            want = np.zeros((2, n, d))
            if newest:
                want[:, max(0, n - m):] = x[b][:, max(0, m - n):]
            else:
                want[:, :min(n, m)] = x[b][:, :n]
            assert np.array_equal(got[b].double().cpu().numpy(), want)


# ----------------------------------------------------------------------- decode

CASES = [
    # lens, H, Hkv, Nq
    ([1], 1, 1, 1),
    ([64], 4, 4, 1),
    ([65, 0, 1], 8, 2, 1),
    ([200, 63], 16, 2, 1),     # 8 rows a kv head
    ([130, 64, 5], 18, 2, 1),  # 9 rows
    ([100, 7], 8, 2, 4),       # 16 rows
    ([3, 0, 150], 4, 2, 8),    # fewer keys than queries
    ([90], 32, 1, 3),          # 96 rows: several row blocks
    ([1000, 10, 333], 6, 3, 2),
]


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens, H, Hkv, Nq", CASES)
def test_decode(lens, H, Hkv, Nq, d, causal):
    cache = ref.make_cache(lens, Hkv, d, seed=len(lens) + H + d)
    q = rand((len(lens), H, Nq, d), H + Nq, 2.0)
    scale = 1 / math.sqrt(d)
    o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    check_attention(o, lse, q, cache, causal, scale, f"{lens} H{H} Hkv{Hkv} Nq{Nq}")


@gpu
@pytest.mark.parametrize("d", [8, 16, 40, 56, 72, 80, 104, 120])
def test_decode_padded_head_sizes(d):
    lens = [77, 0, 300]
    cache = ref.make_cache(lens, 2, d, seed=d)
    q = rand((3, 6, 2, d), d)
    o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), causal=True, scale=0.3)
    check_attention(o, lse, q, cache, True, 0.3, f"d{d}")


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_decode_splits_and_joins(d):
    """One head over many blocks, many short sequences to a block, and both in one batch."""
    for lens, H, Hkv in (([20000], 1, 1), ([30 + 7 * i for i in range(150)], 4, 4), ([12000, 1, 0, 64, 500, 3], 8, 2)):
        cache = ref.make_cache(lens, Hkv, d, seed=len(lens))
        q = rand((len(lens), H, 1, d), 9, 3.0)
        o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), scale=0.1)
        torch.cuda.synchronize()
        check_attention(o, lse, q, cache, False, 0.1, f"{len(lens)} sequences")


@gpu
def test_decode_scales_and_extreme_rows():
    """Tensor scales fold into the scores and the result; queries of very large and very small entries, one
    dominating key, and queries whose group neighbours are not finite."""
    d, lens = 128, [500, 70]
    cache = ref.make_cache(lens, 2, d, seed=4, k_scale=0.02, v_scale=30.0)
    q = rand((2, 8, 1, d), 5)
    q[0, 0] *= 2.0 ** 60
    q[0, 1] *= 2.0 ** -60
    q[0, 2] *= 0
    o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), scale=1e-3, k_scale=0.02, v_scale=30.0)
    keep = [1, 2, 3, 4, 5, 6, 7]  # head 0's scores are of the order of 2^60: one key decides
    qs = q.clone()
    qs[0, 0] = 0
    o2, lse2 = o.clone(), lse.clone()
    z, zl = fa.qcache_decode(qs.cuda(), *dev(*cache), scale=1e-3, k_scale=0.02, v_scale=30.0)
    assert torch.equal(o2[:, keep], z[:, keep]) and torch.equal(lse2[:, keep], zl[:, keep])
    check_attention(z, zl, qs, cache, False, 1e-3, "scales", 0.02, 30.0)
    ks, vs = ref.unpack(*cache, d, 0.02, 30.0)
    s = ks[0][0] @ q[0, 0, 0].double().numpy()
    assert np.abs(o[0, 0, 0].double().cpu().numpy() - vs[0][0][s.argmax()]).max() <= 2.0 ** -8 * 30 * 2688
    q[0, 3, 0, 7], q[1, 4, 0, 0] = float("nan"), float("inf")
    o3, lse3 = fa.qcache_decode(q.cuda(), *dev(*cache), scale=1e-3, k_scale=0.02, v_scale=30.0)
    ok = torch.ones((2, 8), dtype=torch.bool)
    ok[0, 3] = ok[1, 4] = False
    assert torch.equal(o3[ok.cuda()], o[ok.cuda()]) and torch.equal(lse3[ok.cuda()], lse[ok.cuda()])
    assert not torch.isfinite(o3[0, 3]).any() and not torch.isfinite(o3[1, 4]).any()


@gpu
def test_decode_small_weights_of_a_long_cache_count():
    """One key of weight 1 and 40000 of weight 2^-21 each: together 2 % of the sum, and their values are what
    the result is made of."""
    d, n = 64, 40001
    k = torch.zeros((1, 1, n, d))
    k[0, 0, 0, 0] = 6.0
    v = torch.ones((1, 1, n, d))
    v[0, 0, 0] = 0
    cache = run_append(k.to(torch.bfloat16), v.to(torch.bfloat16), [n], d)
    q = torch.zeros((1, 1, 1, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    scale = 21 * math.log(2) / 6
    o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), scale=scale)
    check_attention(o, lse, q, cache, False, scale)


@gpu
def test_decode_into_guards_and_refusals():
    d, lens = 64, [100, 0]
    cache = dev(*ref.make_cache(lens, 2, d, seed=2))
    q = rand((2, 4, 1, d), 1).cuda()
    o, lse = fa.qcache_decode(q, *cache)
    buf = torch.full((q.numel() + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[64:-64].view(q.shape)
    lbuf = torch.full((8 + 8,), 7.0, device="cuda")
    nbytes = fa.qcache_decode_workspace_bytes(2, 4, 2, 1, d, cache[1].shape[1])
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    fa.qcache_decode_into(q, *cache, out, lbuf[4:12].view(2, 4, 1), ws[:nbytes])
    assert torch.equal(out, o) and torch.equal(lbuf[4:12].view(2, 4, 1), lse)
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all() and (lbuf[:4] == 7).all() and (lbuf[12:] == 7).all()
    assert (ws[nbytes:] == 0xFF).all()
    with pytest.raises(fa.FaError):
        fa.qcache_decode_into(q, *cache, out, lse, ws[:nbytes - 16])
    with pytest.raises(ValueError):
        fa.qcache_decode_into(q, *cache, out[:1], lse, ws)
    with pytest.raises(ValueError):
        fa.qcache_decode(q.float(), *cache)
    with pytest.raises(ValueError):
        fa.qcache_decode(rand((2, 4, 1, 128), 1).cuda(), *cache)  # a pool of another head size
    with pytest.raises(fa.FaError):
        fa.qcache_decode(rand((2, 3, 1, d), 1).cuda(), *cache)    # H not a multiple of Hkv
    with pytest.raises(fa.FaError):
        fa.qcache_decode(rand((2, 4, 9, d), 1).cuda(), *cache)    # more than 8 query rows


@gpu
def test_pages_out_of_range_are_skipped_and_reported():
    """A table entry outside the pool, and a length beyond the table: those keys do not exist, the others are
    handled, and the status says so."""
    d, lens = 64, [150, 64]
    pool, table, lens_t = ref.make_cache(lens, 2, d, seed=6)
    q = rand((2, 2, 1, d), 2)
    good, _ = fa.qcache_decode(q.cuda(), *dev(pool, table, lens_t))
    assert fa.check_device_status() == 0
    for bad in (len(pool), -1, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        o, lse = fa.qcache_decode(q.cuda(), *dev(pool, t, lens_t))
        assert fa.check_device_status() == 1 and fa.check_device_status() == 0
        cut = torch.tensor([128, 64], dtype=torch.int32)
        check_attention(o, lse, q, (pool, table, cut), False, 0.125)
        k, v = fa.qcache_read(*dev(pool, t, lens_t), 150, d)
        assert fa.check_device_status() == 1
        assert not k[0, :, 128:].any() and not v[0, :, 128:].any() and k[0, :, :128].any()
        w = fa.qcache_weights(q.cuda(), lse, *dev(pool, t, lens_t), torch.zeros((2, 2, 192), device="cuda"))
        assert fa.check_device_status() == 1
        assert not w[0, :, 128:].any() and w[0, :, :128].all()
        p = pool.cuda()
        fa.qcache_append(*dev(rand((2, 2, 30, d), 1), rand((2, 2, 30, d), 2)), p, *dev(t, lens_t))
        assert fa.check_device_status() == 1
        for page in range(len(pool)):  # only the pages that exist were written
            if page not in (int(table[0, 1]), int(table[1, 0])):
                assert torch.equal(p[page].cpu(), pool[page])
        p = pool.cuda()
        fa.qcache_evict(p, *dev(t, lens_t), torch.rand((2, 2, 192), device="cuda"), 140)
        assert fa.check_device_status() == 1
    long = torch.tensor([100000, 64], dtype=torch.int32)
    o, _ = fa.qcache_decode(q.cuda(), *dev(pool, table, long))
    assert fa.check_device_status() == 1
    neg = torch.tensor([-5, 64], dtype=torch.int32)
    o, lse = fa.qcache_decode(q.cuda(), *dev(pool, table, neg))
    assert fa.check_device_status() == 0
    assert not o[0].any() and (lse[0] == -math.inf).all() and torch.equal(o[1], good[1])


# ---------------------------------------------------------------------- weights

@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("lens, H, Hkv, Nq", CASES)
def test_weights(lens, H, Hkv, Nq, d, causal):
    """Each summand is off by its score's and lse's share (2^-18 of sum |q k|, 2^-22 of |lse|) and 2^-20; the sum over
    rows and the addition in fp32 by 2^-20."""
    cache = ref.make_cache(lens, Hkv, d, seed=len(lens) + H + d)
    B, scale = len(lens), 1 / math.sqrt(d)
    q = rand((B, H, Nq, d), H + Nq, 2.0)
    W = max(lens) + 5
    before = torch.rand((B, Hkv, W), generator=torch.Generator().manual_seed(1))
    dc = dev(*cache)
    _, lse = fa.qcache_decode(q.cuda(), *dc, causal=causal, scale=scale)
    w = fa.qcache_weights(q.cuda(), lse, *dc, before.cuda(), causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    ks, _ = ref.unpack(*cache, d)
    w64, drive = ref.gathered(q, lse, ks, causal, scale, W)
    want = before.double().numpy() + w64
    err = np.abs(w.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -18 * drive + 2.0 ** -20 * want).all(), err.max()
    for b, n in enumerate(lens):
        assert torch.equal(w[b, :, n:].cpu(), before[b, :, n:])
    same = before.cuda()
    fa.qcache_weights(q.cuda(), lse, *dc, same, causal=causal, scale=scale, out=same)
    assert torch.equal(same, w)
    # Every row that saw a key gave away exactly 1.
    rows = (lse.reshape(B, Hkv, -1) > -math.inf).sum(-1).double().cpu()
    got = (w.double().cpu() - before.double()).sum(-1)
    assert ((got - rows).abs() <= 1e-4 * (rows + 1)).all()


@gpu
def test_weights_narrower_than_the_cache():
    d, lens = 64, [300]
    cache = dev(*ref.make_cache(lens, 2, d, seed=1))
    q = rand((1, 2, 1, d), 1).cuda()
    _, lse = fa.qcache_decode(q, *cache)
    wide = fa.qcache_weights(q, lse, *cache, torch.zeros((1, 2, 300), device="cuda"))
    slim = fa.qcache_weights(q, lse, *cache, torch.zeros((1, 2, 101), device="cuda"))
    assert torch.equal(wide[..., :101], slim)


# --------------------------------------------------------------------- eviction

def choose(w, n, keep, sink, recent):
    """The places that stay, by the definition."""
    if n <= keep:
        return list(range(n))
    mid = range(sink, n - recent)
    key = [(-np.inf if np.isnan(w[j]) else w[j]) for j in mid]
    nan_last = sorted(mid, key=lambda j: (np.isnan(w[j]), -key[j - sink], j))
    return list(range(sink)) + sorted(nan_last[:keep - sink - recent]) + list(range(n - recent, n))


def check_evict(lens, Hkv, d, keep, sink, recent, weights, in_place, seed=0):
    cache = ref.make_cache(lens, Hkv, d, seed=seed, spare=2 + len(lens) * -(-keep // 64))
    pool, table, lens_t = cache
    used = set(table[table >= 0].tolist())
    free = [p for p in range(len(pool)) if p not in used]
    need = -(-keep // 64)
    out_t = None if in_place else torch.tensor(free[:len(lens) * need], dtype=torch.int32).reshape(len(lens), need)
    pd, td, ld, wd = dev(pool, table, lens_t, weights)
    ot = None if in_place else out_t.cuda()
    kept, new, w = fa.qcache_evict(pd, td, ld, wd, keep, sink=sink, recent=recent, table_out=ot)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    assert new.tolist() == [min(n, keep) for n in lens] and torch.equal(wd.cpu().view(torch.int32), weights.view(torch.int32))
    ks, vs = ref.unpack(pool, table, lens_t, d)
    k2, v2 = ref.unpack(pd, table if in_place else out_t, new, d)
    for b, n in enumerate(lens):
        m = min(n, keep)
        for h in range(Hkv):
            src = choose(weights[b, h].numpy(), n, keep, sink, recent)
            assert kept[b, h].tolist() == src + [-1] * (keep - m), (b, h)
            assert np.array_equal(k2[b][h], ks[b][h][src]) and np.array_equal(v2[b][h], vs[b][h][src])
            got = w[b, h].cpu().numpy()
            assert np.array_equal(got[:m], weights[b, h].numpy()[src], equal_nan=True) and not got[m:].any()
    if not in_place:  # the former pages are as they were
        for page in used:
            assert torch.equal(pd[page].cpu(), pool[page])
    for page in free:
        if in_place or page not in set(out_t.flatten().tolist()):
            assert torch.equal(pd[page].cpu(), pool[page])


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens, Hkv, d, keep, sink, recent", [
    ([1], 1, 64, 1, 0, 0),
    ([65, 64, 0, 200], 2, 64, 64, 4, 16),
    ([300, 301], 2, 128, 100, 0, 0),
    ([300, 77], 3, 128, 99, 0, 99),     # a window
    ([300, 77], 3, 40, 99, 99, 0),      # a prefix
    ([2000, 130, 1500], 2, 64, 700, 8, 64),
    ([500], 1, 128, 499, 1, 1),
    ([5000, 4999], 1, 64, 1, 0, 0),
    ([3000], 2, 64, 2999, 0, 5),
])
def test_evict(lens, Hkv, d, keep, sink, recent, in_place):
    g = torch.Generator().manual_seed(len(lens) + keep)
    weights = torch.exp(3 * torch.randn((len(lens), Hkv, max(lens)), generator=g))
    check_evict(lens, Hkv, d, keep, sink, recent, weights, in_place)


@gpu
@pytest.mark.parametrize("kind", ["equal", "few values", "signed zeros", "extremes", "negative", "close"])
def test_evict_orders_any_weights(kind):
    g = torch.Generator().manual_seed(5)
    n = 1100
    w = torch.zeros((2, 2, n))
    if kind == "few values":
        w = torch.randint(0, 3, (2, 2, n), generator=g).float()
    elif kind == "signed zeros":
        w = torch.where(torch.rand((2, 2, n), generator=g) < 0.5, -0.0, 0.0)
        w[..., ::100] = 1e-45
    elif kind == "extremes":
        pick = torch.tensor([0.0, float("inf"), float("-inf"), float("nan"), 1e-45, 3e38, -3e38, 1.0])
        w = pick[torch.randint(0, 8, (2, 2, n), generator=g)]
    elif kind == "negative":
        w = torch.randn((2, 2, n), generator=g)
    elif kind == "close":
        w = 1.0 + torch.randint(0, 600, (2, 2, n), generator=g) * 2.0 ** -23
    check_evict([n, n - 1], 2, 64, 400, 3, 30, w, False)


@gpu
def test_evict_with_narrow_weights_and_refusals():
    """Keys from W on weigh 0."""
    d, n, keep = 64, 200, 50
    cache = dev(*ref.make_cache([n], 1, d, seed=1))
    w = torch.full((1, 1, 100), -1.0, device="cuda")
    w[..., 7] = 2.0
    kept, lens, out = fa.qcache_evict(*cache, w, keep)
    assert kept[0, 0].tolist() == [7] + list(range(100, 149)) and lens.tolist() == [50]
    assert out[0, 0].tolist() == [2.0] + [0.0] * 99
    for kw in (dict(keep=0), dict(keep=5, sink=3, recent=3), dict(keep=5, sink=-1)):
        with pytest.raises(ValueError):
            fa.qcache_evict(*cache, w, **kw)
    with pytest.raises(fa.FaError):  # no room for the kept keys
        fa.qcache_evict(*cache, w, 150, table_out=torch.zeros((1, 1), dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------ sizes and failures

@gpu
def test_offsets_beyond_32_bits():
    """Pages whose bytes lie past 4 GB in the pool: append, read, decode, weights and eviction find them."""
    d, Hkv, pages, n = 128, 1, 480000, 200
    pool = torch.empty((pages, Hkv, 9216), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 32
    table = torch.tensor([[pages - 1, 5, pages - 2, 233017], [pages - 3, 466034, 7, pages - 4]], dtype=torch.int32)
    lens = torch.tensor([n, n + 50], dtype=torch.int32)
    k, v = rand((2, Hkv, n, d), 1), rand((2, Hkv, n, d), 2)
    low = torch.empty((8, Hkv, 9216), dtype=torch.uint8, device="cuda")  # the same keys in a small pool
    low_table = torch.arange(8, dtype=torch.int32).reshape(2, 4)
    q = rand((2, 4, 1, d), 3).cuda()
    out = []
    for p, t in ((pool, table), (low, low_table)):
        p[t.flatten().long().cuda()] = 0
        td, ld = dev(t, lens)
        fa.qcache_append(*dev(k, v), p, td, ld)
        o, lse = fa.qcache_decode(q, p, td, ld)
        w = fa.qcache_weights(q, lse, p, td, ld, torch.zeros((2, Hkv, 256), device="cuda"))
        kept, new, w2 = fa.qcache_evict(p, td, ld, w, 90, sink=2, recent=10)
        out.append([o, lse, w, kept, new, w2, *fa.qcache_read(p, td, new, 90, d)])
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert (out[0][3] >= 0).all() and torch.isfinite(out[0][1]).all()


@gpu
@pytest.mark.parametrize("B, d, H", [(33, 64, 2), (257, 64, 2), (2048, 64, 2), (2048, 128, 2), (2048, 64, 9), (2048, 128, 9)])
def test_many_sequences(B, d, H):
    """Batches past a warp, a block and up to the limit (with the shared memory of every kernel instance), with
    empty sequences among them; one more is refused."""
    Hkv = 1
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, 130, B)]
    lens[0], lens[-1] = 0, 129
    cache = ref.make_cache(lens, Hkv, d, seed=B)
    q = rand((B, H, 1, d), B)
    o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), scale=0.2)
    check_attention(o, lse, q, cache, False, 0.2, f"B{B}")
    w = fa.qcache_weights(q.cuda(), lse, *dev(*cache), torch.zeros((B, Hkv, 130), device="cuda"), scale=0.2)
    rows = torch.tensor([H if n else 0 for n in lens], dtype=torch.float64)
    assert ((w.double().sum(-1)[:, 0].cpu() - rows).abs() <= 1e-4).all()
    if B == 2048:
        more = torch.zeros((B + 1, 3), dtype=torch.int32, device="cuda")
        with pytest.raises(fa.FaError):
            fa.qcache_decode(rand((B + 1, H, 1, d), 1).cuda(), cache[0].cuda(), more, more[:, 0].contiguous())


@gpu
@pytest.mark.parametrize("call", ["decode", "weights"])
def test_a_wait_that_runs_out_is_reported_and_recoverable(call):
    """A copy that is never made (test hook): the wait gives up after its limit, the status says so, and the
    next call is right.  No fault, trap or hang is involved."""
    d, lens = 128, [1000, 200]
    cache = ref.make_cache(lens, 2, d, seed=3)
    q = rand((2, 4, 1, d), 1)
    dc = dev(*cache)
    o, lse = fa.qcache_decode(q.cuda(), *dc)
    zero = torch.zeros((2, 2, 1000), device="cuda")
    w = fa.qcache_weights(q.cuda(), lse, *dc, zero)
    assert fa.check_device_status() == 0
    fa.set_wait_limit_ns(20_000_000)  # 20 ms
    fa.debug_skip_k_tile(0)
    try:
        if call == "decode":
            fa.qcache_decode(q.cuda(), *dc)
        else:
            fa.qcache_weights(q.cuda(), lse, *dc, zero)
        torch.cuda.synchronize()
        assert fa.check_device_status() == 4  # FA_ERR_TIMEOUT
    finally:
        fa.debug_skip_k_tile(-1)
        fa.set_wait_limit_ns(0)
    assert fa.check_device_status() == 0
    o2, lse2 = fa.qcache_decode(q.cuda(), *dc)
    w2 = fa.qcache_weights(q.cuda(), lse, *dc, zero)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)
    check_attention(o2, lse2, q, cache, False, 1 / math.sqrt(d))


@gpu
def test_results_do_not_depend_on_timing():
    d = 128
    lens = [5000, 17, 0, 900, 2500]
    cache = dev(*ref.make_cache(lens, 2, d, seed=9))
    q = rand((5, 16, 1, d), 2).cuda()
    first = None
    for _ in range(10):
        o, lse = fa.qcache_decode(q, *cache)
        w = fa.qcache_weights(q, lse, *cache, torch.zeros((5, 2, 5000), device="cuda"))
        kept, new, w2 = fa.qcache_evict(cache[0].clone(), cache[1], cache[2], w, 300, sink=1, recent=9)
        if first is None:
            first = (o, lse, w, kept, new, w2)
        assert all(torch.equal(a, b) for a, b in zip(first, (o, lse, w, kept, new, w2)))


@gpu
def test_evict_longer_heads_than_shared_memory_holds():
    """A head whose weights are read again in each pass, with many equal ones around the border."""
    n = 50000
    g = torch.Generator().manual_seed(1)
    w = torch.randint(0, 40, (1, 1, n), generator=g).float() * 0.25
    check_evict([n], 1, 64, 20000, 3, 100, w, True)


@gpu
def test_numbers_of_any_kind():
    """numpy's numbers are taken as Python's are."""
    d = 64
    cache = dev(*ref.make_cache([100], 2, d, seed=1))
    q = rand((1, 2, 1, d), 1).cuda()
    o, lse = fa.qcache_decode(q, *cache, scale=0.125)
    o2, lse2 = fa.qcache_decode(q, *cache, scale=np.float32(0.125), k_scale=np.float32(1), v_scale=np.float64(1), causal=np.bool_(False))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    w = torch.zeros((1, 2, 128), device="cuda")
    w = fa.qcache_weights(q, lse, *cache, w, scale=np.float32(0.125), k_scale=np.float32(1))
    k, v = fa.qcache_read(*cache, np.int64(10), d, k_scale=np.float32(1))
    assert k.shape == (1, 2, 10, d)
    kept, _, _ = fa.qcache_evict(*cache, w, np.int32(10), sink=np.int64(1), recent=np.int64(2))
    assert kept.shape == (1, 2, 10)
    f, _ = fa.rope_frequencies(d)
    a, _ = fa.rope(q, None, f, factor=np.float32(1.5))
    b, _ = fa.rope(q, None, f, factor=1.5)
    assert torch.equal(a, b)


@gpu
def test_a_page_table_with_much_more_room_than_keys():
    """Only the entries that hold keys are read: the rest of a 16 MB table is out of range everywhere."""
    d, lens = 64, [70, 3]
    pool, table, lens_t = ref.make_cache(lens, 2, d, seed=4)
    wide = torch.full((2, 2_000_000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = rand((2, 4, 1, d), 2).cuda()
    a = fa.qcache_decode(q, *dev(pool, table, lens_t))
    b = fa.qcache_decode(q, *dev(pool, wide, lens_t))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and fa.check_device_status() == 0
    w = [fa.qcache_weights(q, a[1], *dev(pool, t, lens_t), torch.zeros((2, 2, 70), device="cuda")) for t in (table, wide)]
    assert torch.equal(*w)
    r = [fa.qcache_evict(*dev(pool, t, lens_t), w[0], 30) for t in (table, wide)]
    assert torch.equal(r[0][0], r[1][0]) and torch.equal(r[0][2], r[1][2]) and fa.check_device_status() == 0


@gpu
def test_sequences_that_share_pages():
    """A common prefix held once: sequences whose tables begin with the same pages read, attend, gather weights and
    are cut back (into pages of their own) as if each held a copy; appending goes to their own last pages."""
    d, Hkv, n = 64, 2, [200, 170, 200]
    pool, table, lens = ref.make_cache([200, 0, 0], Hkv, d, seed=5, max_pages=4, spare=20)
    free = [p for p in range(len(pool)) if p not in set(table[0].tolist())]
    own = torch.tensor(free[:12], dtype=torch.int32).reshape(3, 4)
    shared = table[0].repeat(3, 1)
    shared[:, 2:] = own[:, :2]          # the first 128 keys are common
    for b in range(3):                  # copies of the rest
        pool[shared[b, 2].long()], pool[shared[b, 3].long()] = pool[table[0, 2].long()], pool[table[0, 3].long()]
    lens = torch.tensor(n, dtype=torch.int32)
    k, v = rand((3, Hkv, 20, d), 1), rand((3, Hkv, 20, d), 2)
    q = rand((3, 4, 1, d), 3).cuda()
    pd, td, ld = dev(pool, shared, lens)
    fa.qcache_append(*dev(k, v), pd, td, ld)
    ks, vs = ref.unpack(pd, td, ld, d)
    for b in range(3):
        assert np.array_equal(ks[b][:, :128], ks[0][:, :128])
        code, byte = ref.quantise(k[b].double().numpy())
        assert np.array_equal(ks[b][:, n[b] - 20:], ref.value(code, byte)[..., :d])
    o, lse = fa.qcache_decode(q, pd, td, ld)
    check_attention(o, lse, q.cpu(), (pd, td, ld), False, 1 / math.sqrt(d))
    w = fa.qcache_weights(q, lse, pd, td, ld, torch.zeros((3, Hkv, 256), device="cuda"))
    out = torch.tensor(free[12:18], dtype=torch.int32).reshape(3, 2).cuda()
    kept, new, _ = fa.qcache_evict(pd, td, ld, w, 90, sink=3, recent=20, table_out=out)
    k2, v2 = ref.unpack(pd, out, new, d)
    assert fa.check_device_status() == 0
    for b in range(3):
        for h in range(Hkv):
            src = choose(w[b, h].cpu().numpy(), n[b], 90, 3, 20)
            assert kept[b, h].tolist() == src
            assert np.array_equal(k2[b][h], ks[b][h][src]) and np.array_equal(v2[b][h], vs[b][h][src])


@gpu
@pytest.mark.parametrize("call", ["decode", "weights"])
def test_many_rows_over_ragged_segments(call):
    """40 and 64 query rows a kv head (several row blocks) over sequences that begin and end inside warps' runs."""
    for d, H, Hkv, Nq, lens in ((64, 16, 2, 5, [700, 3, 0, 64, 1290]), (128, 8, 1, 8, [3000, 65, 1, 400])):
        cache = ref.make_cache(lens, Hkv, d, seed=H)
        q = rand((len(lens), H, Nq, d), 7)
        dc = dev(*cache)
        o, lse = fa.qcache_decode(q.cuda(), *dc, causal=True, scale=0.15)
        if call == "decode":
            check_attention(o, lse, q, cache, True, 0.15, f"{H * Nq // Hkv} rows")
            continue
        W = max(lens) + 1
        before = torch.rand((len(lens), Hkv, W), generator=torch.Generator().manual_seed(2))
        w = fa.qcache_weights(q.cuda(), lse, *dc, before.cuda(), causal=True, scale=0.15)
        same = before.cuda()
        fa.qcache_weights(q.cuda(), lse, *dc, same, causal=True, scale=0.15, out=same)
        assert torch.equal(w, same)
        ks, _ = ref.unpack(*cache, d)
        w64, drive = ref.gathered(q, lse, ks, True, 0.15, W)
        want = before.double().numpy() + w64
        assert (np.abs(w.double().cpu().numpy() - want) <= 2.0 ** -18 * drive + 2.0 ** -20 * want).all()


@gpu
@pytest.mark.parametrize("d", [64, 128, 40, 72])
@pytest.mark.parametrize("H, Hkv, Nq", [(17, 1, 1), (8, 2, 8), (66, 2, 1), (64, 1, 1), (13, 1, 5), (65, 1, 2), (6, 2, 6)])
def test_decode_of_more_rows_than_a_product_takes(H, Hkv, Nq, d):
    """17 to 130 query rows a kv head, whole and partial row blocks, over sequences within a block, across
    blocks, empty, and of one head in many blocks."""
    for lens, causal in (([300, 0, 64, 1, 6000], True), ([20000], False), ([5, 129, 63], True)):
        cache = ref.make_cache(lens, Hkv, d, seed=H + d)
        q = rand((len(lens), H, Nq, d), H, 2.0)
        o, lse = fa.qcache_decode(q.cuda(), *dev(*cache), causal=causal, scale=0.1)
        torch.cuda.synchronize()
        assert fa.check_device_status() == 0
        check_attention(o, lse, q, cache, causal, 0.1, f"{H * Nq // Hkv} rows, {lens}")


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_skip_pages_out_of_range(d):
    lens = [150, 64, 3000]
    pool, table, lens_t = ref.make_cache(lens, 2, d, seed=6)
    q = rand((3, 40, 1, d), 2)
    t = table.clone()
    t[0, 2], t[2, 46] = len(pool), -1
    o, lse = fa.qcache_decode(q.cuda(), *dev(pool, t, lens_t), scale=0.1)
    assert fa.check_device_status() == 1 and fa.check_device_status() == 0
    check_attention(o, lse, q, (pool, table, torch.tensor([128, 64, 46 * 64], dtype=torch.int32)), False, 0.1)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_keep_to_their_own(d):
    """Queries that are not finite reach their own rows alone; values that are not finite reach every row; the
    result is the same each time, and the same rows give the same result among others."""
    lens = [500, 1, 0, 4000]
    pool, table, lens_t = ref.make_cache(lens, 1, d, seed=8)
    q = rand((4, 36, 1, d), 5)
    o, lse = fa.qcache_decode(q.cuda(), *dev(pool, table, lens_t), scale=0.1)
    check_attention(o, lse, q, (pool, table, lens_t), False, 0.1)
    for _ in range(5):
        again = fa.qcache_decode(q.cuda(), *dev(pool, table, lens_t), scale=0.1)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    q2 = q.clone()
    q2[0, 3, 0, 7], q2[3, 20, 0, 0] = float("nan"), float("inf")
    o2, lse2 = fa.qcache_decode(q2.cuda(), *dev(pool, table, lens_t), scale=0.1)
    ok = torch.ones((4, 36), dtype=torch.bool)
    ok[0, 3] = ok[3, 20] = False
    assert torch.equal(o2[ok.cuda()], o[ok.cuda()]) and torch.equal(lse2[ok.cuda()], lse[ok.cuda()])
    assert not torch.isfinite(o2[0, 3]).any() and not torch.isfinite(o2[3, 20]).any()
    few, few_lse = fa.qcache_decode(q[:, :8].contiguous().cuda(), *dev(pool, table, lens_t), scale=0.1)
    check_attention(few, few_lse, q[:, :8], (pool, table, lens_t), False, 0.1)
    x = rand((4, 1, 1, d), 1)
    x[0, 0, 0, 3] = float("nan")
    one = torch.tensor([501, 0, 0, 0], dtype=torch.int32)
    p = pool.cuda()
    fa.qcache_append(*dev(rand((4, 1, 1, d), 2), x), p, *dev(table, one))
    o3, _ = fa.qcache_decode(q.cuda(), p, *dev(table, one), scale=0.1)
    few3, _ = fa.qcache_decode(q[:, :8].contiguous().cuda(), p, *dev(table, one), scale=0.1)
    assert torch.equal(torch.isfinite(o3[0, :8]), torch.isfinite(few3[0]))


@gpu
def test_a_wait_of_many_rows_that_runs_out():
    """As above, with several row blocks a kv head."""
    d, lens = 128, [3000, 200]
    cache = ref.make_cache(lens, 2, d, seed=3)
    q = rand((2, 80, 1, d), 1)
    dc = dev(*cache)
    o, lse = fa.qcache_decode(q.cuda(), *dc)
    assert fa.check_device_status() == 0
    fa.set_wait_limit_ns(20_000_000)  # 20 ms
    fa.debug_skip_k_tile(0)
    try:
        fa.qcache_decode(q.cuda(), *dc)
        torch.cuda.synchronize()
        assert fa.check_device_status() == 4  # FA_ERR_TIMEOUT
    finally:
        fa.debug_skip_k_tile(-1)
        fa.set_wait_limit_ns(0)
    assert fa.check_device_status() == 0
    o2, lse2 = fa.qcache_decode(q.cuda(), *dc)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attention(o2, lse2, q, cache, False, 1 / math.sqrt(d))


@gpu
@pytest.mark.parametrize("newest", [False, True])
def test_read_reports_a_length_beyond_the_table(newest):
    d = 64
    pool, table, lens = ref.make_cache([150, 64], 2, d, seed=6)
    long = torch.tensor([table.shape[1] * 64 + 1, 64], dtype=torch.int32)
    want, _ = fa.qcache_read(*dev(pool, table, lens), 200, d, newest=newest)
    assert fa.check_device_status() == 0
    got, _ = fa.qcache_read(*dev(pool, table, long), 200, d, newest=newest)
    assert fa.check_device_status() == 1 and fa.check_device_status() == 0
    assert torch.equal(got[1], want[1])


@gpu
def test_evict_into_a_narrower_table_at_the_same_address():
    """The destination's rows are entries of the table that hold no key: sequences of at most `keep` keys move too."""
    d, lens, keep = 64, [100, 90], 100
    pool, table, lens_t = ref.make_cache(lens, 2, d, seed=3, max_pages=4, spare=8)
    free = [p for p in range(len(pool)) if p not in set(table[0, :2].tolist()) | set(table[1, :2].tolist())]
    table[0, 2:] = torch.tensor(free[:2], dtype=torch.int32)
    pd, td, ld = dev(pool, table, lens_t)
    out = td.view(-1)[:4].view(2, 2)  # row 1 is row 0's spare entries
    assert out.data_ptr() == td.data_ptr()
    ks, vs = ref.unpack(pool, table, lens_t, d)
    kept, new, _ = fa.qcache_evict(pd, td, ld, torch.rand((2, 2, 100), device="cuda"), keep, table_out=out)
    assert fa.check_device_status() == 0 and new.tolist() == lens
    k2, v2 = ref.unpack(pd, out, new, d)
    for b in range(2):
        assert np.array_equal(k2[b], ks[b]) and np.array_equal(v2[b], vs[b])
        assert kept[b, 0, :lens[b]].tolist() == list(range(lens[b]))
