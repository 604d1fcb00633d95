"""Trees of drafted tokens over the 4-bit cache (fa_qcache_tree) and the commit of the
accepted path (fa_qcache_commit), against the definition in 64 bits.

Attention's bound is that of the cache's decode: a score is off by delta = 2^-18 * big
(big the largest scale * sum |q k|), a probability by its rounding to fp16 (2^-11), the
sums by 2^-20, and the result by its rounding to bf16.  Where one key takes nearly
all of a row's weight and holds 0 in a channel, what the others hold there is all
there is: fp16's smallest step is 2^-24, of probabilities whose largest is at least
2^7, so a weight may be off by half a step, 2^-32 of the largest, whatever its size:
2^-32 * sum |v| over the row's keys (the largest weight being at most 1), and as much
again for the sum that divides it.
"""
import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
import _tree

gpu = pytest.mark.gpu


def dev(*ts):
    return tuple(t.cuda() for t in ts)


def rand(shape, seed, mult=1.0):
    return (torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)) * mult).to(torch.bfloat16)


def trees(B, T, seed):
    return torch.from_numpy(_tree.ancestors(_tree.random_parents(B, T, np.random.default_rng(seed))))


def check(o, lse, q, words, cache, d, scale, k_scale=1.0, v_scale=1.0, rows=slice(None)):
    ks, vs = ref.unpack(*cache, d, k_scale, v_scale)
    o64, lse64, mag, big = _tree.attention(q, words, ks, vs, scale)
    o, lse = o.double().cpu().numpy()[:, :, rows], lse.double().cpu().numpy()[:, :, rows]
    o64, lse64, mag, big = (x[:, :, rows] for x in (o64, lse64, mag, big))
    delta = 2.0 ** -18 * big
    most = np.zeros((len(ks), o64.shape[1], 1, 1))  # a bound on sum |v| of every head
    for b, v in enumerate(vs):
        if v.shape[1]:
            most[b] = np.repeat(np.abs(v).sum(1).max(-1), o64.shape[1] // v.shape[0])[:, None, None]
    bound = 2.0 ** -8 * np.abs(o64) + (2.0 ** -11 + 2.0 ** -20 + 2 * delta[..., None]) * mag + 2.0 ** -31 * most
    err = np.abs(o - o64)
    assert (err <= bound).all(), f"o: {(err / np.where(bound > 0, bound, 1e-30)).max():.2f} of the bound"
    gone = np.isneginf(lse64)
    assert (np.isneginf(lse) == gone).all()
    err = np.abs(np.where(gone, 0, lse) - np.where(gone, 0, lse64))
    assert (err <= delta + 2.0 ** -19 * (1 + np.abs(np.where(gone, 0, lse64)))).all(), f"lse off by {err.max():.2e}"


def run(q, words, cache, scale=None, **more):
    o, lse = fa.qcache_tree(q.cuda(), words.cuda(), *dev(*cache), scale=scale, **more)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    return o, lse


# ------------------------------------------------------------- words and depths

@pytest.mark.parametrize("T", [1, 2, 7, 63, 64])
def test_tree_words(T):
    parents = _tree.random_parents(5, T, np.random.default_rng(T))
    words, depths = fa.tree_words(torch.from_numpy(parents))
    want = _tree.ancestors(parents)
    assert np.array_equal(words.numpy(), want)
    assert np.array_equal(depths.numpy(), np.array([[bin(int(w) & (2 ** 64 - 1)).count("1") - 1 for w in row] for row in want]))
    one, _ = fa.tree_words(torch.from_numpy(parents[0]))
    assert torch.equal(one, words[0])


def test_tree_words_refuses():
    for bad in (torch.tensor([0, 0]), torch.tensor([-1, 2, 0]), torch.zeros(0, dtype=torch.int64), torch.zeros(65, dtype=torch.int64) - 1,
                torch.tensor([-1.0]), torch.zeros((1, 1, 1), dtype=torch.int64)):
        with pytest.raises(ValueError):
            fa.tree_words(bad)


# --------------------------------------------------------------------- attention

# Drafts around page borders: alone in the cache, ending a page, starting one, over two pages.
@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T, lens, H, Hkv", [
    (1, [1, 64, 65, 700], 4, 2), (3, [3, 64, 66, 130], 2, 2), (8, [8, 72, 64, 400, 127], 8, 2), (17, [17, 100, 64], 4, 4),
    (64, [64, 65, 127, 128, 700], 4, 2), (33, [2000, 33, 64], 14, 2), (21, [500, 97], 16, 1), (5, [5000], 4, 4),
    (64, [300, 129], 8, 1), (13, [129, 128, 257], 40, 4)])
def test_trees(T, lens, H, Hkv, d):
    cache = ref.make_cache(lens, Hkv, d, seed=T)
    q, words = rand((len(lens), H, T, d), T + d), trees(len(lens), T, T)
    o, lse = run(q, words, cache)
    check(o, lse, q, words, cache, d, d ** -0.5)


@gpu
@pytest.mark.parametrize("d", [8, 40, 56, 72, 104, 120])
def test_padded_head_sizes(d):
    lens = [200, 64, 31]
    cache = ref.make_cache(lens, 2, d, seed=d)
    for T in (4, 30):
        q, words = rand((3, 6, T, d), d), trees(3, T, d)
        o, lse = run(q, words, cache)
        check(o, lse, q, words, cache, d, d ** -0.5)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T, H", [(2, 2), (12, 4), (64, 4)])
def test_rows_that_see_nothing_and_sequences_shorter_than_the_tree(T, H, d):
    """Empty words over an empty context, drafts of negative position, sequences without keys."""
    lens = [T, T + 70, max(1, T // 2), 0, 1]
    cache = ref.make_cache(lens, 2, d, seed=T, max_pages=3)
    words = trees(5, T, 3)
    words[:, ::2] = 0
    q = rand((5, H, T, d), 4)
    o, lse = run(q, words, cache)
    check(o, lse, q, words, cache, d, d ** -0.5)
    assert (o[0, :, ::2] == 0).all() and torch.isneginf(lse[0, :, ::2]).all() and (o[3] == 0).all()


@gpu
@pytest.mark.parametrize("T", [5, 40])
def test_any_set_of_drafts(T):
    """Words that are no trees, with bits beyond the drafts, which stand for no key."""
    lens = [300, 64, 130]
    cache = ref.make_cache(lens, 2, 128, seed=1)
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (3, T), generator=torch.Generator("cpu").manual_seed(2))
    q = rand((3, 8, T, 128), 3)
    o, lse = run(q, words, cache)
    check(o, lse, q, words, cache, 128, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("T, H", [(7, 2), (40, 4)])
def test_padded_drafts_hold_anything(T, H):
    """Drafts that no word names: their keys, values and queries reach no other row."""
    B, d, n = 2, 64, 90
    words, real = trees(B, T, 13), T - 3
    words[:, real:] = 0
    q, k, v = rand((B, H, T, d), 14), rand((B, 2, n, d), 15), rand((B, 2, n, d), 16)
    pool, table = fa.qcache_pool(6, 2, d), torch.arange(6, dtype=torch.int32, device="cuda").reshape(B, 3).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    fa.qcache_append(k.cuda(), v.cuda(), pool, table, lens)
    want = fa.qcache_tree(q.cuda(), words.cuda(), pool, table, lens)
    for i, x in enumerate((float("nan"), float("inf"), -3e38)):
        k[:, :, n - 3 + i], v[:, :, n - 3 + i], q[:, :, real + i] = x, x, x
    fa.qcache_append(k.cuda(), v.cuda(), pool, table, lens)
    got = fa.qcache_tree(q.cuda(), words.cuda(), pool, table, lens)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    assert torch.isfinite(want[0]).all()
    for a, b in zip(got, want):
        # (The rows may be scaled by powers of two of their own, which changes no rounding of
        # queries above 2^-31 of the largest: all of them.)
        assert torch.equal(a[:, :, :real], b[:, :, :real])


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 4, 8])
def test_a_chain_is_causal_decode(Nq, d):
    lens = [70, 500, 64 + Nq]
    cache = dev(*ref.make_cache(lens, 2, d, seed=6))
    q = rand((3, 4, Nq, d), 7).cuda()
    words, depths = fa.tree_words(torch.arange(Nq, device="cuda").expand(3, Nq) - 1)
    assert depths.tolist() == [list(range(Nq))] * 3
    o, lse = fa.qcache_tree(q, words.contiguous(), *cache)
    o2, lse2 = fa.qcache_decode(q, *cache, causal=True)
    # Two roundings to bf16 of sums that differ by 2^-18 of sum p |v|.
    assert ((o.float() - o2.float()).abs() <= 2.0 ** -7 * o2.float().abs() + 2.0 ** -10).all()
    assert ((lse - lse2).abs() <= 2.0 ** -17 * (1 + lse2.abs())).all()


@gpu
@pytest.mark.parametrize("T, H", [(3, 2), (30, 4)])
def test_scales_and_large_scores(T, H):
    k_scale, v_scale = 0.37, 2.0 ** -3
    lens = [333, 90]
    cache = ref.make_cache(lens, 2, 128, seed=8, k_scale=k_scale, v_scale=v_scale, gain=3.0)
    q, words = rand((2, H, T, 128), 9, 30.0), trees(2, T, 9)
    q[:, :, -1] *= 2.0 ** -90
    o, lse = run(q, words, cache, scale=0.2, k_scale=k_scale, v_scale=v_scale)
    check(o, lse, q, words, cache, 128, 0.2, k_scale, v_scale)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T, H", [(5, 2), (9, 2), (12, 4), (30, 4), (64, 4)])
@pytest.mark.parametrize("B, powers", [(3, (0, -12)), (3, (-110, -30, -16, 0, 3, 18)), (90, (-110, -30, -16, 0, 3, 18))])
def test_queries_of_unequal_size(B, powers, T, H, d):
    """Rows far apart in size share a product, each as exact as if it were alone, and rows
    that hold NaN, infinities or the largest numbers leave the others as they are."""
    rng = np.random.default_rng(T + B)
    lens = [int(n) for n in rng.integers(T, T + 250, B)]
    cache = ref.make_cache(lens, 2, d, seed=T)
    words = trees(B, T, 11)
    q = rand((B, H, T, d), 12) * torch.from_numpy(2.0 ** rng.choice(powers, (B, H, T, 1))).to(torch.bfloat16)
    o, lse = run(q, words, cache)
    check(o, lse, q, words, cache, d, d ** -0.5)
    bad = q.clone()
    bad[:, :, 1], bad[:, :, 2], bad[:, :, 3] = float("nan"), float("inf"), torch.finfo(torch.bfloat16).max
    o, lse = run(bad, words, cache)
    check(o, lse, q, words, cache, d, d ** -0.5, rows=[i for i in range(T) if i not in (1, 2, 3)])


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B, H, T, n", [(1, 4, 20, 30000), (1, 64, 64, 5000), (300, 2, 9, 90), (40, 4, 33, 700)])
def test_long_and_many(B, H, T, n, d):
    """Work split over many blocks, and over many sequences; parts joined."""
    rng = np.random.default_rng(B)
    lens = [n] + [int(x) for x in rng.integers(0, n + 1, B - 1)]
    cache = ref.make_cache(lens, 2, d, seed=B, max_pages=-(-n // 64))
    q, words = rand((B, H, T, d), B + 1), trees(B, T, B)
    o, lse = run(q, words, cache)
    check(o, lse, q, words, cache, d, d ** -0.5)


@gpu
@pytest.mark.parametrize("T", [4, 40])
def test_pages_beyond_32_bits(T):
    """A pool of more than 2^32 bytes, its last pages in use."""
    d, lens = 128, [150, T + 64]
    pool, table, n = ref.make_cache(lens, 2, d, seed=T)
    pages, first = pool.shape[0], (1 << 32) // (2 * 9216) + 5
    wide = torch.empty((first + pages, 2, 9216), dtype=torch.uint8, device="cuda")
    wide[first:] = pool.cuda()
    q, words = rand((2, 4, T, d), T), trees(2, T, 5)
    small, large = dev(pool, table, n), (wide, (table + first).to(torch.int32).cuda(), n.cuda())
    for a, b in zip(fa.qcache_tree(q.cuda(), words.cuda(), *small), fa.qcache_tree(q.cuda(), words.cuda(), *large)):
        assert torch.equal(a, b)
    path = torch.tensor([[1, 3], [0, 2]], dtype=torch.int32, device="cuda")
    assert torch.equal(fa.qcache_commit(*small, path, T), fa.qcache_commit(*large, path, T))
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    assert torch.equal(small[0], wide[first:])


@gpu
@pytest.mark.parametrize("T, H", [(4, 4), (48, 4)])
def test_pages_and_lengths_out_of_range_are_skipped_and_reported(T, H):
    lens = [300, 200]
    pool, table, n = ref.make_cache(lens, 2, 128, seed=11)
    q, words = rand((2, H, T, 128), 12), trees(2, T, 12)
    good_o, good_lse = run(q, words, (pool, table, n))
    bad = table.clone()
    bad[0, 1] = len(pool) + 5
    o, lse = fa.qcache_tree(q.cuda(), words.cuda(), *dev(pool, bad, n))
    assert fa.check_device_status() == 1
    assert torch.equal(o[1], good_o[1]) and torch.equal(lse[1], good_lse[1])
    # The page's keys are skipped: the same as a sequence without them, its words on the same drafts.
    ks, vs = ref.unpack(pool, table, n, 128)
    keep = np.r_[0:64, 128:300]
    o64, lse64, mag, big = _tree.attention(q[:1], words[:1], [ks[0][:, keep]], [vs[0][:, keep]], 128 ** -0.5)
    err = np.abs(o[:1].double().cpu().numpy() - o64)
    assert (err <= 2.0 ** -8 * np.abs(o64) + (2.0 ** -11 + 2.0 ** -20 + 2.0 ** -17 * big[..., None]) * mag).all()
    # A length beyond the table: what the table holds is read, drafts stay where the length puts them.
    n2 = torch.tensor([300, 4 * 64 + 64 + 5], dtype=torch.int32)
    table2 = torch.cat([table, torch.full((2, 1), -1, dtype=torch.int32)], 1)[:, :5].contiguous()
    table2[:, 4] = table[:, 4] if table.shape[1] > 4 else table[0, 0]
    table2[1] = table2[0]
    o, lse = fa.qcache_tree(q.cuda(), words.cuda(), *dev(pool, table2, n2))
    assert fa.check_device_status() == 1
    assert torch.isfinite(o[0].float()).all()


@gpu
def test_into_guards_streams_and_graphs():
    d, T, lens = 128, 24, [200, 90, 24]
    cache = dev(*ref.make_cache(lens, 2, d, seed=13, max_pages=6))
    q, words = rand((3, 4, T, d), 14).cuda(), trees(3, T, 14).cuda()
    want_o, want_lse = fa.qcache_tree(q, words, *cache)
    obuf = torch.full((q.numel() + 128,), -77.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((3 * 4 * T + 128,), -77.0, device="cuda")
    o, lse = obuf[64:-64].view(q.shape), lbuf[64:-64].view(3, 4, T)
    need = fa.qcache_tree_workspace_bytes(3, 4, 2, T, d, 6)
    ws = torch.full((need + 128,), 77, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.qcache_tree_into(q, words, *cache, o, lse, ws[64:-64], stream=side)
    side.synchronize()
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
    for b, f in ((obuf, -77.0), (lbuf, -77.0), (ws, 77)):
        assert (b[:64] == f).all() and (b[-64:] == f).all()
    with torch.cuda.stream(side):
        fa.qcache_tree(q, words, *cache)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.qcache_tree(q, words, *cache)
    cache[2].copy_(torch.tensor([130, 64, 80], dtype=torch.int32))
    # Pages of the second and third sequences reach no further than before.
    cache[2][1:] = torch.tensor([90, 24], dtype=torch.int32)
    words.copy_(trees(3, T, 15))
    graph.replay()
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    check(o, lse, q.cpu(), words.cpu(), tuple(t.cpu() for t in cache), d, d ** -0.5)


@gpu
@pytest.mark.parametrize("T", [4, 40])
def test_a_wait_that_runs_out_is_reported(T):
    cache = ref.make_cache([5000, 900], 2, 128, seed=16)
    q, words = rand((2, 4, T, 128), 17), trees(2, T, 17)
    want = run(q, words, cache)
    fa.set_wait_limit_ns(20_000_000)
    try:
        fa.debug_skip_k_tile(0)  # the first warp may have no second page
        fa.qcache_tree(q.cuda(), words.cuda(), *dev(*cache))
        assert fa.check_device_status() == 4
    finally:
        fa.debug_skip_k_tile(-1)
        fa.set_wait_limit_ns(0)
    got = run(q, words, cache)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------ commit

def rows_of(cache, d):
    ks, vs = ref.unpack(*cache, d)
    return [np.stack([k, v]) for k, v in zip(ks, vs)]


@gpu
@pytest.mark.parametrize("d", [64, 128, 24])
@pytest.mark.parametrize("T, lens, paths", [
    (1, [1, 64, 65], [[0], [-1], [0]]),
    (8, [8, 64, 70, 129, 127], [[0, 1, 2], [7, -1, -1], [1, 3, 5], [-1, -1, -1], [0, 2, 7]]),
    (64, [64, 100, 128, 700], [[63] + [-1] * 8, list(range(1, 18, 2)), list(range(9)), [0, 5, 9, 10, 33, 34, 62, 63, -1]]),
    (64, [200, 65], [list(range(64)), list(range(1, 64)) + [-1]]),
    (33, [97, 96, 40], [list(range(0, 33, 2)), list(range(16, 33)), [32] + [-1] * 16]),
    (6, [4, 0, 6], [[2, 5], [-1, -1], [4, 5]])])
def test_commit(T, lens, paths, d):
    pool, table, n = ref.make_cache(lens, 2, d, seed=T, max_pages=13)
    path = torch.tensor(paths, dtype=torch.int32)
    before = rows_of((pool, table, n), d)
    gp, gt, gn = dev(pool, table, n)
    got = fa.qcache_commit(gp, gt, gn, path.cuda(), T)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    want_lens, touched = [], torch.zeros(pool.shape, dtype=torch.bool)
    keep = []
    for b, m in enumerate(lens):
        first = max(m - T, 0)
        kept = [i + m - T for i in paths[b] if i >= 0]
        want_lens.append(first + len(kept))
        keep.append(np.concatenate([before[b][:, :, :first], before[b][:, :, kept]], 2))
    assert got.tolist() == want_lens
    after = rows_of((gp.cpu(), table, got.cpu()), d)
    for b in range(len(lens)):
        assert np.array_equal(after[b], keep[b]), b
    # Nothing but the path's new places changes.
    D = ref.stored_channels(d)
    kc, ks, vc, vs = ref.places(D)
    changed = (gp.cpu() != pool).numpy()
    may = np.zeros(pool.shape, bool)
    for b, m in enumerate(lens):
        first = max(m - T, 0)
        for x in range(first, want_lens[b]):
            page, r = int(table[b, x // 64]), x % 64
            for where in (kc, ks, vc, vs):
                may[page][:, where[r]] = True
    assert not (changed & ~may).any()
    # Of a byte that two keys share only the new key's half changes.
    for b, m in enumerate(lens):
        first, end = max(m - T, 0), want_lens[b]
        for x in (first - 1, end):  # neighbours in the same byte
            if x < 0 or x // 2 not in (first // 2, (end - 1) // 2) or first == end or x // 64 >= table.shape[1]:
                continue
            page, r = int(table[b, x // 64]), x % 64
            if page < 0:
                continue
            sh = 4 * (r % 2)
            assert np.array_equal(gp[page].cpu().numpy()[:, vc[r]] >> sh & 15, pool[page].numpy()[:, vc[r]] >> sh & 15)


@gpu
def test_commit_ends_and_reports_at_what_is_no_path():
    """Not rising, beyond the drafts, a draft that the sequence does not hold; an end is no error."""
    T, lens = 8, [100, 100, 100, 5, 100]
    pool, table, n = dev(*ref.make_cache(lens, 2, 64, seed=3))
    for row, bad, count in ((0, [3, 3, 4], 1), (1, [2, 8, 9], 1), (2, [5, 1, 6], 1), (3, [2, 4, 5], 0), (4, [-5, 3, 4], 0)):
        path = torch.full((5, 3), -1, dtype=torch.int32)
        path[row] = torch.tensor(bad)
        got = fa.qcache_commit(pool.clone(), table, n, path.cuda(), T)
        assert fa.check_device_status() == (0 if row == 4 else 1)
        want = [92, 92, 92, 0, 92]
        want[row] += count
        assert got.tolist() == want, row


@gpu
def test_commit_skips_and_reports_pages_out_of_range():
    T = 70 - 64 + 10
    pool, table, n = ref.make_cache([70], 2, 64, seed=4)
    bad = table.clone()
    bad[0, 1] = len(pool)
    gp = pool.cuda()
    got = fa.qcache_commit(gp, bad.cuda(), n.cuda(), torch.tensor([[1, 2, T - 1]], dtype=torch.int32, device="cuda"), T)
    assert fa.check_device_status() == 1 and got.tolist() == [70 - T + 3]
    spare = [p for p in range(len(pool)) if p != int(table[0, 0])]
    assert torch.equal(gp.cpu()[spare], pool[spare])


@gpu
def test_commit_follows_values_in_a_graph_and_streams():
    T = 8
    pool, table, n = dev(*ref.make_cache([100, 77], 2, 128, seed=5))
    path = torch.tensor([[1, 4, -1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = fa.qcache_commit(pool.clone(), table, n, path, T, stream=side)
    side.synchronize()
    assert out.tolist() == [94, 70]
    torch.cuda.current_stream().wait_stream(side)
    work = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.qcache_commit(work, table, n, path, T)
    path.copy_(torch.tensor([[7, -1, -1], [2, 3, 5]], dtype=torch.int32))
    work.copy_(pool)
    graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [93, 72]
    want = pool.clone()
    assert fa.qcache_commit(want, table, n, path, T).tolist() == [93, 72]
    assert torch.equal(want, work) and fa.check_device_status() == 0


# -------------------------------------------------------------- a run of them

@gpu
@pytest.mark.parametrize("T, H, Hkv, d", [(7, 4, 2, 64), (40, 8, 2, 128)])
def test_verifying_steps(T, H, Hkv, d):
    """Draft, turn by depth, append, attend by the tree, cross attention, commit: three
    steps, the cache always that of the accepted tokens alone, as one key at a time makes it."""
    B, Nk = 2, 150
    rng = np.random.default_rng(20)
    freqs, factor = fa.rope_frequencies(d)
    pool, plain = fa.qcache_pool(40, Hkv, d), fa.qcache_pool(40, Hkv, d)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(B, 20).contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    plain_lens = lens.clone()
    states_k, states_v = (torch.randn((B, Hkv, Nk, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    for step in range(3):
        parents = torch.from_numpy(_tree.random_parents(B, T, rng)).cuda()
        words, depths = fa.tree_words(parents)
        positions = (lens[:, None] + depths).to(torch.int32).contiguous()
        q, k, v = (rand((B, h, T, d), 100 * step + i).cuda() for i, h in enumerate((H, Hkv, Hkv)))
        q, k = fa.rope(q, k, freqs, positions=positions, factor=factor)
        lens = lens + T
        fa.qcache_append(k, v, pool, table, lens)
        o, lse = fa.qcache_tree(q, words, pool, table, lens)
        check(o, lse, q.cpu(), words.cpu(), tuple(t.cpu() for t in (pool, table, lens)), d, d ** -0.5)
        c, _ = fa.cross_fwd(o, states_k, states_v)
        s = d ** -0.5 * torch.einsum("bhnd,bhmd->bhnm", o.double(), states_k.double().repeat_interleave(H // Hkv, 1))
        want = torch.softmax(s, -1) @ states_v.double().repeat_interleave(H // Hkv, 1)
        assert (c.double() - want).abs().max() <= 2.0 ** -6 * want.abs().max() + 2.0 ** -7
        # The deepest draft's path is accepted.
        leaf = depths.argmax(-1)
        path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            w = int(words[b, leaf[b]]) & (2 ** 64 - 1)
            kept = [j for j in range(T) if w >> j & 1]
            path[b, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
            # The accepted tokens' rows one at a time, turned at the places they have come to.
            for j in kept:
                plain_lens[b] += 1
                one = torch.where(torch.arange(B, device="cuda") == b, plain_lens, 0).to(torch.int32)
                fa.qcache_append(k[:, :, j:j + 1].contiguous(), v[:, :, j:j + 1].contiguous(), plain, table, one)
        lens = fa.qcache_commit(pool, table, lens, path, T)
        assert torch.equal(lens, plain_lens)
        n = int(lens.max())
        for a, b in zip(fa.qcache_read(pool, table, lens, n, d), fa.qcache_read(plain, table, plain_lens, n, d)):
            assert torch.equal(a, b)
    assert fa.check_device_status() == 0
