"""A length beyond its page table: keys that have no page do not exist, and each query still
sees the keys up to its own position (lens[b] - Nq + i), not up to one counted from the table's end."""
import math

import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
from test_qcache import check_attention, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H, Nq", [(2, 4), (6, 8)])
@pytest.mark.parametrize("over", [1, 2, 7, 1000, 2 ** 31 - 1 - 128])
@pytest.mark.parametrize("d", [64, 128])
def test_causal_queries_past_the_table(d, over, H, Nq):
    held, Hkv = 128, 2
    pool, table, lens = ref.make_cache([held, 40], Hkv, d, seed=d)
    q = rand((2, H, Nq, d), 3)
    scale = 1 / math.sqrt(d)
    said = lens.clone()
    said[0] = held + over
    o, lse = fa.qcache_decode(q.cuda(), pool.cuda(), table.cuda(), said.cuda(), causal=True, scale=scale)
    w = fa.qcache_weights(q.cuda(), lse, pool.cuda(), table.cuda(), said.cuda(), torch.zeros((2, Hkv, held), device="cuda"),
                          causal=True, scale=scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 1 and fa.check_device_status() == 0  # reported once
    # Query i stands at key said - Nq + i: with `over` keys missing it sees min(held, said - Nq + i + 1).
    for i in range(Nq):
        n = min(held, held + over - Nq + i + 1)
        one = torch.tensor([n, max(0, 40 - Nq + i + 1)], dtype=torch.int32)
        check_attention(o[:, :, i:i + 1], lse[:, :, i:i + 1], q[:, :, i:i + 1], (pool, table, one), False, scale, f"query {i}")
    # Every query's weights sum to one.
    total = w.double().sum(-1).cpu().numpy()
    assert np.allclose(total, H // Hkv * Nq, rtol=1e-4)
