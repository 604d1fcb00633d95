"""Cosine and sine of rotary positions to their own size: where one member of a pair is zero
the other's share is the whole result, however small the angle or its distance from a quarter turn.

Bound.  The angle is an integer multiple of 2^-64 of a turn, taken to the nearest quarter turn exactly; what is left
becomes fp32 (2^-24 of itself), its series stops at 2^-24 of the value, its Horner steps round five times (2^-24 each
of the largest term, at most 1.4 times the value), and the factor and the product round once each (2 * 2^-24):
below 10 * 2^-24 < 2^-20 of the result.  Then the result's rounding to bf16: 2^-8 of it.
"""
import math

import pytest
import torch

import io_aware_attention_gb300 as fa

pytestmark = pytest.mark.gpu


def exact(pos, words):
    """cos and sin of pos * word in 64 bits: the product modulo one turn in whole numbers, then to the nearest quarter
    turn, so that small values keep their digits."""
    out = torch.empty((2, len(pos), len(words)), dtype=torch.float64)
    for i, t in enumerate(pos):
        for j, w in enumerate(words):
            a = (t * w) % 2 ** 64
            quarter, r = divmod(a + 2 ** 61, 2 ** 62)
            x = (r - 2 ** 61) / 2 ** 64 * 2 * math.pi
            c, s = math.cos(x), math.sin(x)
            for _ in range(quarter % 4):
                c, s = -s, c
            out[0, i, j], out[1, i, j] = c, s
    return out


def close(got, want):
    got, want = got.double().cpu(), want
    err = (got - want).abs()
    assert (err <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all(), f"off by {(err / want.abs().clamp(min=1e-300)).max().item():.3e} of the result"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d, rot", [(128, 128), (64, 64), (80, 36), (80, 38)])
@pytest.mark.parametrize("stretch", [1.0, 8.0])
def test_each_member_alone(d, rot, layout, stretch):
    """Pairs (a, 0) and (0, b): four products, each against its own size; forward and gradient."""
    freqs, _ = fa.rope_frequencies(rot, scaling="linear" if stretch > 1 else "none", factor=stretch, device="cpu")
    words = [w % 2 ** 64 for w in freqs.tolist()]
    pos = [0, 1, 2, 3, 5, 17, 100, 4095, -1, -2, 10 ** 6, 2 ** 31 - 1]
    N = len(pos)
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    g = torch.Generator("cpu").manual_seed(rot)
    x = torch.randn((1, 6, N, rot // 2), generator=g).to(torch.bfloat16)
    c, s = exact(pos, words)
    at = torch.tensor(pos, dtype=torch.int64).cuda()
    factor = 1.25
    for inverse in (False, True):
        s_ = -s if inverse else s
        for first in (True, False):
            q = torch.zeros((1, 6, N, d), dtype=torch.bfloat16)
            q[..., one if first else two] = x
            got, _ = fa.rope(q.cuda(), None, freqs.cuda(), positions=at, layout=layout, factor=factor, inverse=inverse)
            v = x.double() * factor
            close(got[..., one], v * c if first else -v * s_)
            close(got[..., two], v * s_ if first else v * c)
            assert not got[..., rot:].any()


def test_near_quarter_turns_and_at_far_positions():
    """Frequency words of 1 and beside each quarter turn, and positions up to 2^62: the product is the integer's."""
    words = [1, 2 ** 20, 2 ** 62 - 1, 2 ** 62 + 1, 2 ** 63 - 3, 2 ** 63 + 2 ** 30, 2 ** 64 - 1, 3 * 2 ** 62 - 2 ** 25, 2 ** 61, 2 ** 61 - 1,
             5 * 2 ** 61, 12345678901234567890, 1 << 40, (1 << 64) - (1 << 41), 2 ** 62, 2 ** 63]
    pos = [1, 3, -1, 2 ** 45 + 1, -(2 ** 50) - 7, 2 ** 62 + 5]
    freqs = torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64)
    c, s = exact(pos, words)
    d, N = 2 * len(words), len(pos)
    for first in (True, False):
        q = torch.zeros((1, 2, N, d), dtype=torch.bfloat16)
        half = slice(0, d // 2) if first else slice(d // 2, d)
        q[..., half] = 1.5
        got, _ = fa.rope(q.cuda(), None, freqs.cuda(), positions=torch.tensor(pos).cuda())
        close(got[..., :d // 2], 1.5 * (c if first else -s).expand(1, 2, N, -1))
        close(got[..., d // 2:], 1.5 * (s if first else c).expand(1, 2, N, -1))
