"""rope_into on views that share a buffer but no place: one-token views of a fused projection,
views by heads of one tensor, and views by batch; on the CPU up to the device check, on the GPU
against the same call on copies."""
import itertools

import pytest
import torch

import io_aware_attention_gb300 as fa

from test_rope import rand
from test_serve_abi import P, lib, needs_lib, rope  # noqa: F401  (lib is a fixture)


def places(offset, s, B, H, N, d):
    return {offset + b * s[0] + h * s[1] + n * s[2] + c for b in range(B) for h in range(H) for n in range(N) for c in range(d)}


# (queries' strides, keys' strides, keys' offset in elements, B, H, Hk, N): all in one buffer, no place in common.
APART = [
    ((192, 64, 64), (192, 64, 64), 128, 3, 2, 1, 1),       # (B, (H + Hk) d) projection seen as (B, H, 1, d)
    ((192, 64, 192), (192, 64, 192), 128, 3, 2, 1, 1),     # the same by transposed views
    ((256, 64, 128), (256, 64, 192), 128, 3, 2, 1, 1),     # strides over one position differ and mean nothing
    ((320, 64, 64), (320, 64, 64), 0 + 192, 2, 2, 2, 1),   # with a gap between
    ((640, 128, 64), (640, 128, 64), 256, 2, 2, 1, 2),     # (B, heads, N, d): queries' heads, then keys'
    ((1280, 128, 64), (1280, 128, 64), 640, 2, 2, 1, 2),   # halves of a batch's row
    ((64, 384, 192), (64, 384, 192), 1536, 3, 2, 2, 2),    # batches interleave, heads apart
    ((1024, 64, 256), (1024, 64, 256), 128, 2, 2, 2, 4),   # fused projection of four positions
    ((0, 64, 192), (0, 64, 192), 128, 1, 2, 1, 5),         # one batch: its stride means nothing
    ((768, 0, 192), (768, 0, 192), 64, 2, 1, 1, 4),        # one head: its stride means nothing
]
# The same with places in common.
SHARED = [
    ((192, 64, 64), (192, 64, 64), 64, 3, 2, 1, 1),
    ((192, 64, 64), (192, 64, 64), 160, 3, 2, 1, 1),
    ((128, 64, 64), (128, 64, 64), 128, 3, 2, 1, 1),       # the keys of a batch are the next one's queries
    ((640, 128, 64), (640, 128, 64), 64, 2, 2, 1, 2),
    ((1280, 128, 64), (1280, 128, 64), 1280, 2, 2, 1, 2),
    ((1024, 64, 256), (1024, 64, 256), 64, 2, 2, 2, 4),
]


def test_the_cases_are_what_they_say():
    for cases, shared in ((APART, False), (SHARED, True)):
        for qs, ks, at, B, H, Hk, N in cases:
            q, k = places(0, qs, B, H, N, 64), places(at, ks, B, Hk, N, 64)
            assert len(q) == B * H * N * 64 and len(k) == B * Hk * N * 64 and bool(q & k) == shared


@needs_lib
@pytest.mark.parametrize("case", APART)
def test_views_apart_are_accepted(lib, case):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would run on fake addresses")
    qs, ks, at, B, H, Hk, N = case
    for a, b in ((0, 2 * at), (2 * at, 0)):  # the queries before the keys, and after them
        if b == 0:
            qs, ks, H, Hk = ks, qs, Hk, H
        kw = dict(q=P + a, k=P + b, qs=qs, ks=ks, B=B, H=H, Hk=Hk, N=N)
        assert rope(lib, qo=P + a, ko=P + b, qos=qs, kos=ks, **kw) in (2, 3)   # in place (2, 3: no device)
        assert rope(lib, qo=5 * P + a, ko=5 * P + b, qos=qs, kos=ks, freqs=9 * P, **kw) in (2, 3)  # into another such buffer


@needs_lib
@pytest.mark.parametrize("case", SHARED)
def test_views_that_share_places_are_refused(lib, case):  # noqa: F811
    qs, ks, at, B, H, Hk, N = case
    kw = dict(q=P, k=P + 2 * at, qs=qs, ks=ks, B=B, H=H, Hk=Hk, N=N)
    assert rope(lib, qo=P, ko=P + 2 * at, qos=qs, kos=ks, **kw) == 1


@needs_lib
def test_no_pair_that_shares_a_place_is_accepted(lib):  # noqa: F811
    """Every small arrangement of two views of 8 channels: where the outputs share a place the call is refused."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would run on fake addresses")
    steps = [0, 4, 8, 12, 16, 24, 40]
    refused = accepted = 0
    for B, H, Hk, N in ((2, 1, 1, 1), (2, 2, 1, 1), (2, 1, 2, 2), (1, 2, 2, 2)):
        for s in itertools.product(steps, repeat=3):
            q = places(0, s, B, H, N, 8)
            if len(q) != B * H * N * 8:
                continue
            for at in (0, 4, 8, 12, 16, 20, 32, 48):
                status = rope(lib, q=7 * P, k=8 * P, qo=P, ko=P + 2 * at, qos=s, kos=s, B=B, H=H, Hk=Hk, N=N, d=8, rot=8)
                if q & places(at, s, B, Hk, N, 8):
                    assert status == 1, (s, at, B, H, Hk, N)
                    refused += 1
                else:
                    accepted += status in (2, 3)
    assert refused > 100 and accepted > 100


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", APART)
def test_views_in_place(case, layout):
    qs, ks, at, B, H, Hk, N = case
    d = 64
    freqs, factor = fa.rope_frequencies(d, device="cuda")
    buf = rand((4096,), 7).cuda()
    q, k = buf.as_strided((B, H, N, d), (*qs, 1)), buf.as_strided((B, Hk, N, d), (*ks, 1), at)
    pos = torch.arange(N, device="cuda") + 1000
    want = fa.rope(q.clone(), k.clone(), freqs, positions=pos, layout=layout)
    before = buf.clone()
    fa.rope_into(q, k, q, k, freqs, positions=pos, layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    mine = torch.zeros(4096, dtype=torch.bool, device="cuda")
    mine.as_strided((B, H, N, d), (*qs, 1))[:] = True
    mine.as_strided((B, Hk, N, d), (*ks, 1), at)[:] = True
    assert torch.equal(buf[~mine], before[~mine])
