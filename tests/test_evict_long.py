"""Eviction past what a block's shared memory holds (the weights that do not fit are read
again in every pass) and moves of more pages than one round takes, against a stable sort."""
import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref

pytestmark = pytest.mark.gpu


def chosen(w, n, keep, sink, recent):
    """The kept places of one head by a stable sort of its n weights, largest first."""
    if n <= keep:
        return np.arange(n)
    mid = np.arange(sink, n - recent)
    order = mid[np.argsort(-w[mid], kind="stable")][:keep - sink - recent]
    return np.concatenate([np.arange(sink), np.sort(order), np.arange(n - recent, n)])


@pytest.mark.parametrize("n, Hkv", [(140001, 1), (200000, 3), (131073, 2)])
def test_selection_past_shared_memory(n, Hkv):
    """Clusters of 4 blocks hold 4 * 32768 weights of a head; the places beyond are read again.  Few distinct weights,
    so that most passes tie and the border runs through every block."""
    d, keep, sink, recent = 8, 5000, 10, 300
    pages = -(-n // 64)
    pool = torch.zeros((pages, Hkv, 72 * 64), dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    g = torch.Generator("cpu").manual_seed(n)
    w = torch.randint(0, 40, (1, Hkv, n), generator=g).float() / 8 - 1
    w[:, 0] = torch.randn(n, generator=g)
    kept, new, wo = fa.qcache_evict(pool, table, lens, w.cuda(), keep, sink=sink, recent=recent)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0 and new.tolist() == [keep]
    for h in range(Hkv):
        want = chosen(w[0, h].numpy(), n, keep, sink, recent)
        assert np.array_equal(kept[0, h].cpu().numpy(), want)
        assert torch.equal(wo[0, h, :keep].cpu(), w[0, h][torch.from_numpy(want)]) and not wo[0, h, keep:].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", [False, True])
def test_moves_of_many_rounds(d, apart):
    """8 blocks of 4 pages are a round: 5000 kept keys are 79 pages, three rounds, in place and to other pages."""
    lens, Hkv, keep = [9000, 5100], 2, 5000
    g = torch.Generator("cpu").manual_seed(d)
    most = -(-max(lens) // 64)
    D = ref.stored_channels(d)
    pool = torch.randint(0, 119, (2 * most + 160, Hkv, 72 * D), generator=g, dtype=torch.uint8).cuda()  # no NaN scale
    order = torch.randperm(len(pool), generator=g).to(torch.int32)
    table = order[:2 * most].reshape(2, most).cuda()
    out = order[2 * most:2 * most + 158].reshape(2, 79).cuda() if apart else None
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = fa.qcache_read(pool, table, n, max(lens), d)
    w = torch.rand((2, Hkv, max(lens)), generator=g)
    kept, new, _ = fa.qcache_evict(pool, table, n, w.cuda(), keep, sink=4, recent=50, table_out=out)
    k2, v2 = fa.qcache_read(pool, table if out is None else out, new, keep, d)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    for b in range(2):
        for h in range(Hkv):
            want = chosen(w[b, h].numpy(), lens[b], keep, 4, 50)
            assert np.array_equal(kept[b, h].cpu().numpy(), want)
    at = kept.long()[..., None].expand(2, Hkv, keep, d)
    assert torch.equal(k2, k.gather(2, at)) and torch.equal(v2, v.gather(2, at))


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_that_stays_is_not_written(d):
    """At most `keep` keys and the table itself: the pages keep every byte, also behind the last key; copied to other
    pages, the places behind the last key are cleared."""
    lens, Hkv, keep = [100, 70, 0], 2, 100
    pool, table, n = (t.cuda() for t in ref.make_cache(lens, Hkv, d, seed=d, spare=8))
    before = pool.clone()
    w = torch.rand((3, Hkv, 128), device="cuda")
    kept, new, wo = fa.qcache_evict(pool, table, n, w, keep)
    torch.cuda.synchronize()
    assert torch.equal(pool, before) and new.tolist() == lens
    assert kept[0, 0].tolist() == list(range(100)) and kept[1, 1].tolist() == list(range(70)) + [-1] * 30
    used = set(table[0, :2].tolist() + table[1, :2].tolist())
    free = [i for i in range(len(pool)) if i not in used]
    out = torch.tensor([free[:2], free[2:4], free[4:6]], dtype=torch.int32, device="cuda")
    fa.qcache_evict(pool, table, n, w, keep, table_out=out)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    full = torch.full_like(n, 128)
    for b, m in enumerate(lens[:2]):
        k, v = fa.qcache_read(pool, out[b:b + 1].contiguous(), full[:1], 128, d)
        k0, v0 = fa.qcache_read(before, table[b:b + 1].contiguous(), n[b:b + 1], 128, d)
        assert torch.equal(k, k0) and torch.equal(v, v0) and not k[:, :, m:].any()
