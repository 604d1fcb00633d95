"""Cross attention of a batch: a sequence's results are its own, and one without keys gives 0 and
-infinity (the sign too), whole, split, captured."""
import math

import pytest
import torch

import io_aware_attention_gb300 as fa

from test_cross import device_lens, draw, run_all

pytestmark = pytest.mark.gpu


# One query row over a split key range, a whole one, and queries in parts.
@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("H, Hkv, Nq, Nk, split", [(2, 2, 1, 2000, True), (8, 2, 70, 333, False), (4, 1, 300, 90, False)])
def test_other_sequences_do_not_matter(d, H, Hkv, Nq, Nk, split):
    """The same number of sequences; the others' rows and lengths change, the kept one's results do not."""
    B, keep = 5, 3
    lens = [Nk, 17, 0, Nk - 29, Nk // 2]
    assert (fa.cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d) > 0) == split
    first = draw(B, H, Hkv, Nq, Nk, d, lens, 50 + d)
    a = run_all(*first, lens)
    lens2 = [1, 0, Nk, lens[keep], 130 % Nk]
    second = draw(B, H, Hkv, Nq, Nk, d, lens2, 51 + d, mult=3.0)
    for x, y in zip(first, second):
        y[keep] = x[keep]
    b = run_all(*second, lens2)
    for name in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[name][keep], b[name][keep]), name


def nothing_seen(o, lse):
    return (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d", [64, 128, 48])
@pytest.mark.parametrize("Nq, Nk", [(1, 3001), (70, 300), (600, 64)])
def test_no_key_gives_minus_infinity(d, Nq, Nk):
    lens = [Nk, 0, 1, 0]
    q, k, v, do = draw(4, 4, 2, Nq, Nk, d, lens, 60 + d)
    got = run_all(q, k, v, do, lens)
    n = device_lens([0] * 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.cross_fwd(q, k, v, n)
    graph.replay()
    torch.cuda.synchronize()
    assert nothing_seen(o, lse)
    n.copy_(device_lens([Nk, -5, 1, 0]))  # (keys behind these hold NaN)
    graph.replay()
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    assert nothing_seen(o[1::2], lse[1::2]) and torch.isfinite(lse[::2]).all()
    for b in (1, 3):
        assert nothing_seen(got["o"][b], got["lse"][b]) and (got["dq"][b] == 0).all()
    for b in (0, 2):
        assert math.isfinite(got["lse"][b].abs().max().item())
