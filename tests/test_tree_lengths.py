"""Drafted trees where the cache holds less than a length says: a length beyond the page table, and a page
outside the pool.  What is left is compared with the definition on the keys that are there."""
import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
from test_tree import check, rand, trees

pytestmark = pytest.mark.gpu


# Few rows a kv head (the decode kernel's form) and many; drafts that the table holds in part, all and none of.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T, H", [(4, 4), (4, 2), (48, 4), (20, 2), (64, 4)])
@pytest.mark.parametrize("over", [1, 2, 70, 4000])
def test_a_length_beyond_the_page_table(T, H, d, over):
    """Drafts stay where the length puts them; those behind the table's last key are seen by none."""
    held = 320
    lens = [300, held + over]
    pool, table, n = ref.make_cache(lens, 2, d, seed=T)
    q, words = rand((2, H, T, d), T), trees(2, T, T)
    o, lse = fa.qcache_tree(q.cuda(), words.cuda(), pool.cuda(), table[:, :held // 64].contiguous().cuda(), n.cuda())
    assert fa.check_device_status() == 1
    there = held - (lens[1] - T)  # drafts that the table holds
    want = words.clone()
    if there > 0:
        want[1] &= (1 << there) - 1
    else:  # every row sees all keys that are held
        n = torch.tensor([300, held], dtype=torch.int32)
        want[1] = -1
    check(o, lse, q, want, (pool, table, n), d, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T, H", [(4, 4), (48, 4), (20, 2)])
@pytest.mark.parametrize("slot", [0, 1, 3])
def test_a_page_outside_the_pool(T, H, d, slot):
    """Its keys are skipped: the same as a cache without them (none of them a draft)."""
    lens = [310, 200]
    pool, table, n = ref.make_cache(lens, 2, d, seed=T + slot)
    q, words = rand((2, H, T, d), T), trees(2, T, T)
    for page in (len(pool), -1, 2 ** 31 - 1):
        bad = table.clone()
        bad[0, slot] = page
        o, lse = fa.qcache_tree(q.cuda(), words.cuda(), pool.cuda(), bad.cuda(), n.cuda())
        assert fa.check_device_status() == 1
        without = table.clone()
        without[0, slot:-1] = table[0, slot + 1:]
        check(o, lse, q, words, (pool, without, torch.tensor([lens[0] - 64, lens[1]], dtype=torch.int32)), d, d ** -0.5)
