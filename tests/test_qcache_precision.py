"""The 4-bit cache's attention where its result is a small difference of large terms: a
rounding of the probabilities shows there, and nowhere else this plainly.

Keys come in pairs whose values are x and -x, and scores are small, so that the weights of a
pair nearly cancel: |o| is far below sum p |v|.

Bound.  A probability 2^(y + 15), y <= 0, is off by its argument's rounding (half a step of 2^-20 below 16,
times ln 2: 2^-21.5), the exponential's 2^-22 and, held as the sum of two fp16 numbers, by 2^-23: below 2^-20
together, and once more in the sum that divides it, so 2^-19.  Its score is off by delta = 2^-18 * big (the bound of
the scores' sums, see test_qcache.py), in the numerator and the denominator.  A group of 16 keys takes two products
onto the accumulator, each with one sum inside and one onto it: four roundings of 2^-23 of sum p |v|, that is 2^-21
a group, and as much again to join pieces.  Then the result's rounding to bf16: 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref

pytestmark = pytest.mark.gpu


def paired_cache(lens, Hkv, d, seed):
    """A cache whose values of keys 2j and 2j + 1 are x and -x."""
    g = torch.Generator("cpu").manual_seed(seed)
    most = max(lens)
    k = torch.randn((len(lens), Hkv, most, d), generator=g).to(torch.bfloat16)
    v = torch.randn((len(lens), Hkv, most, d), generator=g).to(torch.bfloat16)
    v[:, :, 1::2] = -v[:, :, 0::2][:, :, :most // 2]
    pages = -(-most // 64)
    pool = fa.qcache_pool(len(lens) * pages, Hkv, d)
    table = torch.arange(len(lens) * pages, dtype=torch.int32, device="cuda").reshape(len(lens), pages)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    full = torch.full_like(n, most)
    fa.qcache_append(k.cuda(), v.cuda(), pool, table, full)
    return pool, table, n


@pytest.mark.parametrize("d", [64, 128, 40])
@pytest.mark.parametrize("lens, H, Hkv, Nq", [([2, 4], 4, 2, 1), ([2, 64, 6], 16, 1, 1), ([4, 130], 4, 2, 8), ([2], 24, 1, 2),
                                              ([8, 0, 2, 3000], 8, 8, 1)])
def test_probabilities_are_not_rounded_away(lens, H, Hkv, Nq, d):
    cache = paired_cache(lens, Hkv, d, seed=H + d)
    q = torch.randn((len(lens), H, Nq, d), generator=torch.Generator("cpu").manual_seed(Nq)).to(torch.bfloat16)
    scale = 2.0 ** -10
    o, lse = fa.qcache_decode(q.cuda(), *cache, scale=scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    ks, vs = ref.unpack(*cache, d)
    o64, lse64, mag, big = ref.attention(q, ks, vs, False, scale)
    groups = (np.array(lens)[:, None, None, None] + 15) // 16
    bound = 2.0 ** -8 * np.abs(o64) + (2.0 ** -19 + 2.0 ** -17 * big[..., None] + 2 * groups * 2.0 ** -21) * mag
    err = np.abs(o.double().cpu().numpy() - o64)
    assert (err <= bound).all(), f"off by {(err / np.where(bound > 0, bound, 1)).max():.2f} of the bound"
