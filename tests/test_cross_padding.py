"""Cross attention's padding, whatever the queries and the output gradient hold:
gradients of rows behind the last key are zero."""
import math

import pytest
import torch

import io_aware_attention_gb300 as fa

from _cross import check, reference
from test_cross import device_lens, draw, run_all

pytestmark = pytest.mark.gpu


# Key blocks of 128: whole ones, one that holds the last key, ones without a key.  One block
# of queries a head, which is not cut into parts, and several, which are.
@pytest.mark.parametrize("d", [64, 128, 40])
@pytest.mark.parametrize("H, Hkv, Nq, parts", [(2, 2, 40, False), (8, 2, 300, True)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_padding_has_no_gradient_whatever_the_rows_hold(d, H, Hkv, Nq, parts, what):
    """NaN and infinities of dO (sequence 0) and of q (sequence 1): 0 * NaN reaches no padding."""
    lens, Nk = [150, 5, 0, 70], 300
    q, k, v, do = draw(4, H, Hkv, Nq, Nk, d, lens, 40 + d)
    clean = run_all(q, k, v, do, lens)
    need = 4 * H * -(-Nq // 64) * 64 * ((64 if d <= 64 else 128) + 2) * 4
    assert (fa.cross_bwd_workspace_bytes(4, H, Hkv, Nq, Nk, d) > need) == parts
    do[0, :, Nq // 2] = what
    q[1, :, Nq - 1, 0] = what
    got = run_all(q, k, v, do, lens)
    for b, n in enumerate(lens):
        for name in ("dk", "dv"):
            assert (got[name][b, :, n:] == 0).all(), (name, b)
    for b in (2, 3):
        for name in ("o", "lse", "dk", "dv"):
            assert torch.equal(got[name][b], clean[name][b]), (name, b)
    # dq: fp32 sums in an order of their own.
    want = reference(q[2:], k[2:], v[2:], lens[2:], d ** -0.5, do[2:])
    check(got["dq"][2:], want["dq"], "dq")
